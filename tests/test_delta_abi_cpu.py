"""The gated delta rule's C entry points where sequences are counted, on the CPU
(nothing is launched)."""
import ctypes

import pytest

from test_block_cpu import ALIAS, FAKE, GB, _at, _mod
from test_delta_cpu import _delta, _dgrads


def test_no_offsets_and_no_number_of_sequences_are_one():
    """offsets NULL with num_seqs 0 is one sequence of all rows: the same checkpoints
    and workspaces as for 1."""
    b, L = _mod()
    import device_wide_prefix_chained_amd as dw
    n = dw.ps_gated_delta_checkpoint_floats
    for tokens in (0, 1, 64, 65, 1 << 20):
        assert n(tokens, 0, 2, 16, 8) == n(tokens, 1, 2, 16, 8) > 0
    need = [ctypes.c_size_t(0), ctypes.c_size_t(0)]
    for seqs in (0, 1):
        assert L.ps_gated_delta(None, ctypes.byref(need[seqs]), _delta(b, num_seqs=seqs), None, None, None, None) == 0
    assert need[0].value == need[1].value


@pytest.mark.parametrize("seqs", [0, 1])
def test_overlaps_of_the_one_sequences_states_are_refused(seqs):
    """final, initial, dfinal, dinitial and the checkpoints have the sizes of one sequence."""
    b, L = _mod()
    big = ctypes.byref(ctypes.c_size_t(GB))
    arrays = {n: _at(i + 1) for i, n in enumerate(("q", "k", "v", "g", "beta", "initial"))}
    outs = dict(out=_at(10), final=_at(11), checkpoints=_at(12))

    def forward(at):
        return L.ps_gated_delta(FAKE, big, _delta(b, num_seqs=seqs, **{n: at[n] for n in arrays}), at["out"], at["final"],
                                at["checkpoints"], None)
    place = dict(arrays, **outs)
    pairs = [("final", o) for o in place if o != "final"] + [("initial", o) for o in outs] + \
            [("checkpoints", o) for o in place if o != "checkpoints"]
    for name, other in pairs:
        assert forward(dict(place, **{name: place[other] + 8})) == ALIAS, (name, other)
        assert forward(dict(place, **{other: place[name] + 8})) == ALIAS, (name, other)
    grads = {n: _at(20 + i) for i, n in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dinitial"))}
    ins = dict(arrays, dout=_at(13), dfinal=_at(14), checkpoints=_at(12))

    def backward(at):
        return L.ps_gated_delta_bwd(FAKE, big, _delta(b, num_seqs=seqs, **{n: at[n] for n in arrays}), at["dout"],
                                    at["dfinal"], at["checkpoints"], _dgrads(b, **{n: at[n] for n in grads}), None)
    place = dict(ins, **grads)
    pairs = [("dinitial", o) for o in place if o != "dinitial"] + \
            [(n, o) for n in ("initial", "dfinal", "checkpoints") for o in grads]
    for name, other in pairs:
        assert backward(dict(place, **{name: place[other] + 8})) == ALIAS, (name, other)
        assert backward(dict(place, **{other: place[name] + 8})) == ALIAS, (name, other)
