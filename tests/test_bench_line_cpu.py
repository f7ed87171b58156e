"""Host-side check of bench.py's result line: a row's record is short enough that the
line with every row can be read from the last 9 KB of the output."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_rows_record_is_short():
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    import bench
    rec = dict(workload="adamw_bf16p_bf16_sr_1g", format="bf16_sr", optimizer="grad-norm", p_dtype="bf16-sr", elements=6738411520, tensors=290,
               bytes_per_element=12.0625, steps=70, ms_per_step=2.104678916931152, ms_median=2.0985119342803955, ms_p10=2.0789520740509033,
               ms_p90=2.1185500621795654, gelem_per_s=510.16894565829114, achieved_GBps=6170.6830139764415, frac_of_peak=0.7713353767470552,
               launch_ms=2.0989590167999266, host_us_median=9.701999999833788, samples_ms=[2.1186] * 70, round_medians_ms=[2.0945] * 7, rounds=7)
    row = bench.brief(rec)
    assert len(json.dumps(row)) < 320 and 16 * 320 + 3500 < 9000
    for k in ("ms_per_step", "ms_median", "ms_p10", "ms_p90", "gelem_per_s", "achieved_GBps", "frac_of_peak"):
        assert abs(row[k] - rec[k]) <= 5e-6 * rec[k]
    assert row["workload"] == rec["workload"] and row["elements"] == rec["elements"] and row["steps"] == 70
