"""The benchmark's line on standard output: one JSON object with the headline's keys, short enough for a log's tail
(which held 8 KB and some of standard error where it was recorded whole, and cut lines of 12 KB and more)."""
import json

import bench

PARITY = dict(ids_bit_exact=True, offsets_bit_exact=True, weights_max_rel=2.5411665809658235e-07,
              out_rel_l2=0.0012142081339354739, out_max_rel=0.005649717514124294, tokens_compared=128, within_bar=True,
              bar="ids/offsets bit-exact; weights 1e-6 relative; out rel-L2 <= 2e-3, max|d| <= 1e-2 max|ref|")
SPREAD = dict(median=0.5983033499999735, p10=0.5883033499999735, p90=0.6083033499999735)


def cpu():
    return dict(value=32.37208210577113, unit="tokens/s", cores=16, kind="oracle", seconds=11.862072965999998, repetitions=3,
                cpu_model="AMD EPYC 9575F 64-Core Processor", sample="routing/quantisation/permutation of all 19647 tokens, "
                "expert FFN + combine of 16 evenly spaced tokens, 1 times; rate = those tokens / wall time", parity=PARITY)


def workload(name):
    roof = dict(bound="mfma", achieved=1977.9401372138886, peak=5000.0, unit="TFLOP/s", frac=0.3955880274427777)
    return dict(workload=name, T=19647, H=4096, I=2048, E=256, topk=8, activation="relu2 (gate-less)", routing="learned + zipf bias",
                ms_per_step=2.487982900000052, tokens_per_s=3292627.1318021636, ffn_ms=1.9549834489822389, active_experts=256,
                load_max_over_mean=1.3515625, idle_experts=0, weight_bytes=3424124928, ffn_flop=3298534883328,
                ffn_hbm_gbs=1751.4853794709072, ffn_tflops=1687.2444035499182, roofline_hbm=roof, roofline_mfma=roof,
                deterministic=True, step_device_ms=SPREAD, ffn_device_ms=SPREAD,
                cold_cache=dict(scratch_bytes=536870912, step_device_ms=SPREAD, ffn_device_ms=SPREAD, tokens_per_s=3292627.1318021636),
                attribution_ms=dict(route=0.0281234567, permute=0.0112345678, expert_ffn=0.5412345678, combine=0.0091234567),
                power_clock=dict(power_w_mean=1234.567890123, power_w_max=1399.0, sclk_mhz_mean=2123.456789, sclk_mhz_max=2400.0,
                                 samples=123, seconds=1.0123456789), roofline=roof, cpu_baseline=cpu())


def record():
    roof = dict(workload("decode")["roofline"], traffic=3403705789.0, traffic_unit="HBM bytes per FFN (rocprofv3 FETCH_SIZE + "
                "WRITE_SIZE, copy-calibrated)", algorithmic_bytes=3370622976, kernel="k_ffn_persistent (expert FFN: both grouped "
                "GEMMs, SwiGLU, requant, scatter)", kernel_ms=0.540350404381752)
    rec = dict(metric=bench.METRIC, value=213938.29735368467, unit="tokens/s", n_gpus=1, steps=20, warmup=5,
               ms_per_step=0.5983033499999735, higher_is_better=True, scaling="weak", vs_baseline=None, dtype="fp8e4m3",
               data="synthetic", config=dict(workload="decode", T=128, H=4096, I=2048, E=256, topk=8, activation="swiglu",
                                             weights="fp4-e2m1/e8m0-32/fp32-128x128", parallelism="none (one GPU)"),
               roofline=roof, cpu_baseline=cpu(), parity=PARITY, deterministic=True, detail=workload("decode"))
    for k in ("prefill", "zipf", "hash", "ragged", "tiny"):
        rec[k] = workload(k)
    rec["weight_quantizer"] = dict(E=256, H=4096, I=2048, weights=6442450944, ms=5.4531234567, algorithmic_bytes=29193404416,
                                   bound="hbm", achieved=5354.1234567, peak=8000.0, unit="GB/s", frac=0.6692654321,
                                   kernel="k_quantize_weights (fp32 master -> packed fp4 e2m1 + e8m0 + fp32 block scale)")
    rec["backward"] = [dict(workload=w, T=8192, ms=19.670123456, p10=19.48, p90=19.757, tokens_per_s=416471.23456,
                            algorithmic_bytes=32883499008, bf16_flops=6597069766656, hbm_frac=0.2089, bf16_mfma_frac=0.1341,
                            ideal_ms_hbm=4.11, ideal_ms_bf16_mfma=2.64, bound="hbm", achieved=1671.23456, peak=8000.0,
                            unit="GB/s", frac=0.2089123456) for w in ("decode", "prefill")]
    rec["gateless"] = [workload(w) for w in ("decode_relu2", "prefill_relu2")]
    return rec


def test_short_and_whole():
    rec = record()
    text = bench.line(rec)
    assert len(text) < 6000 and "\n" not in text
    assert len(json.dumps(rec)) > 12000          # what it is taken from
    got = json.loads(text)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
              "dtype", "data", "config", "roofline", "parity", "deterministic"):
        assert got[k] == rec[k]
    assert abs(got["prefill"]["tokens_per_s"] / rec["prefill"]["tokens_per_s"] - 1) < 1e-5
    assert got["ragged"]["parity"]["within_bar"] and got["backward"][1]["workload"] == "prefill"
    assert json.loads(json.dumps(rec)) == json.loads(json.dumps(record()))          # the record itself is left alone


def test_without_side_records():
    rec = record()
    for k in ("prefill", "zipf", "hash", "ragged", "tiny", "weight_quantizer", "backward", "gateless"):
        del rec[k]
    rec["cpu_baseline"] = rec["parity"] = None
    rec["detail"].update(cold_cache=None, attribution_ms=None, power_clock=None)
    assert json.loads(bench.line(rec))["value"] == rec["value"]
    assert "OUTSIDE" in bench.parity_text(dict(PARITY, within_bar=False)) and "DIFFER" in bench.parity_text(dict(PARITY, ids_bit_exact=False))
