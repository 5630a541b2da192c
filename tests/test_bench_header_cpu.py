"""bench.py ties a counter summary to what its kernel uses of the public header, and
the committed summaries are those of the present kernels."""
import json
import os
import re

import pytest

from test_bench_cpu import ROOT, bench

SUMMARIES = sorted(f[len("traffic_"):-len(".json")] for f in os.listdir(os.path.join(ROOT, "profiles"))
                   if re.fullmatch(r"traffic_.*\.json", f))


def _header():
    with open(os.path.join(ROOT, "include", "dwps.h"), encoding="utf-8") as f:
        return bench._without_comments(f.read())


@pytest.mark.parametrize("workload", SUMMARIES)
def test_committed_summaries_are_of_these_sources(workload):
    with open(os.path.join(ROOT, "profiles", "traffic_%s.json" % workload)) as f:
        assert bench.load_traffic(workload, 1.0) == float(json.load(f)["hbm_bytes_per_launch"])


def test_every_declaration_is_found_once():
    found = [n for n, _ in bench._declarations(_header())]
    assert len(found) == len(set(found))
    for name in ("PS_WS_HEADER_BYTES", "PS_WS_MAGIC", "PS_F16", "PS_STREAM_READ", "ps_scan", "ps_scan_input", "ps_delta_grads",
                 "ps_gated_delta_step", "ps_layer_norm_bwd", "ps_status_string"):
        assert name in found, name
    # every name with our prefix that stands before a bracket is a function, and found
    code = " ".join(_header().split())
    assert set(re.findall(r"\b(ps_\w+)\s*\(", code)) <= set(found)


def test_declarations_for_other_kernels_do_not_count():
    header = _header()
    used = lambda h: bench.used_declarations(h, {"ps_scan", "PS_ERR_SIZE"})  # noqa: E731
    want = used(header)
    assert "ps_scan(" in want and "PS_ERR_SIZE = 3" in want and "ps_gated_delta" not in want
    # what ps_scan's types name comes with it only where it has a text of its own
    more = header.replace("const char *ps_version(void);", "#define PS_OTHER 3\ntypedef struct ps_other {\n    int a, b;\n} ps_other;\n"
                          "ps_status ps_other_call(const ps_other *in);\nconst char *ps_version(void);")
    assert more != header and used(more) == want
    assert used(header.replace("PS_F16 = 4", "PS_F16 = 4, PS_F64 = 5")) == want
    # a change to what is used is one
    assert used(header.replace("PS_ERR_SIZE = 3", "PS_ERR_SIZE = 13")) != want
    assert used(header.replace("ps_status ps_scan(void *ws,", "ps_status ps_scan(const void *ws,")) != want
    # a struct's members count where a function that is used takes it
    layer = lambda h: bench.used_declarations(h, {"ps_layer_norm"})  # noqa: E731
    assert "ps_layer_input" in layer(header)
    assert layer(header.replace("const float *weight, *bias;", "const float *bias, *weight;")) != layer(header)
