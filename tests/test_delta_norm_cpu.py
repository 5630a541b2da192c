"""What the norms of delta_norm tell apart, on the CPU: the formulas of a chunk agree
with the rule token by token, and with a term left out, a sign turned or one fp16
plane in the place of two every result is refused."""
import pytest
import torch

import delta_chunks
import delta_norm
import delta_ref as ref

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

CASES = [  # tokens, cuts, kheads, heads, key_dim, value_dim, type, normalize, initial
    (200, None, 2, 2, 64, 64, BF16, True, True),
    (200, [0, 50, 190], 2, 4, 40, 36, F16, True, True),
    (190, [0, 50, 190], 1, 2, 128, 130, BF16, False, True),
    (150, None, 1, 3, 33, 17, F32, True, True),
    (130, [0, 66, 130], 1, 2, 256, 40, F32, True, True),
    (1000, [3, 1000], 1, 1, 32, 24, BF16, True, True),
]


def inputs(case):
    """As the GPU's tests make them."""
    T, cuts, KH, H, K, V, dtype, normalize, initial = case
    g = torch.Generator().manual_seed(T + K)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731

    def keys():
        v = r(T, KH, K)
        return (v if normalize else 0.9 * v / v.norm(dim=-1, keepdim=True)).to(dtype)
    seqs = 1 if cuts is None else len(cuts) - 1
    a = dict(q=keys(), k=keys(), v=r(T, H, V).to(dtype), g=delta_norm.decays(T, H, g),
             beta=torch.sigmoid(r(T, H)), normalize=normalize, initial=0.5 * r(seqs, H, K, V) if initial else None,
             offsets=None if cuts is None else torch.tensor(cuts), dout=r(T, H, V).to(dtype),
             dfinal=0.3 * r(seqs, H, K, V) if initial else None)
    return a, slice(0, T) if cuts is None else slice(cuts[0], cuts[-1])


def kind_of(name, dtype):
    return dtype if name in ("out", "dq", "dk", "dv") else F32


def refused(name, got, want, dtype):
    try:
        delta_norm.close(name, got.to(kind_of(name, dtype)), want)
    except AssertionError:
        return True
    return False


def parts(res, rows):
    return {n: t if n in ("final", "dinitial") else t[rows] for n, t in res.items()}


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norms_tell_mistakes(case):
    a, rows = inputs(case)
    want = parts(ref.delta(**a, dtype=case[6])[0], rows)
    got = parts(delta_chunks.delta(**a), rows)
    assert set(want) == set(got) == set(delta_chunks.TERMS)
    for name, w in want.items():
        assert float((got[name] - w).norm()) <= 1e-11 * float(w.norm()), name
        assert not refused(name, w, w, case[6])
        assert refused(name, torch.zeros_like(w), w, case[6]) and refused(name, -w, w, case[6]), name
        one = w.clone()
        one[one.shape[0] // 2, 0] = 0.0  # of one head, a row or a state
        assert refused(name, one, w, case[6]), name
    for name, terms in delta_chunks.TERMS.items():
        for term in terms:
            bad = parts(delta_chunks.delta(**a, drop=term), rows)
            assert refused(name, bad[name], want[name], case[6]), (name, term)


@pytest.mark.parametrize("case", [c for c in CASES if c[6] != F32], ids=str)
def test_norms_tell_one_plane_from_two(case):
    """In 16-bit calls: every fp32 result and, of those of 16 bits, out."""
    a, rows = inputs(case)
    want = parts(ref.delta(**a, dtype=case[6])[0], rows)
    two, one = (parts(delta_chunks.delta(**a, planes=n), rows) for n in (2, 1))
    for name in want:
        assert not refused(name, two[name], want[name], case[6]), name
    for name in ("out", "final", "dinitial", "dg", "dbeta"):
        assert refused(name, one[name], want[name], case[6]), name


def test_half_a_step():
    for kind in (BF16, F16, F32):
        v = torch.tensor([1.0, 1.75, 2.0, -3.0, 0.4, 1e-3, 0.0], dtype=torch.float64)
        above = torch.nextafter(v.to(kind).abs(), torch.tensor(float("inf"), dtype=kind)).double()
        assert torch.equal(2 * delta_norm.half_step(kind, v.to(kind).double())[:-1], (above - v.to(kind).double().abs())[:-1])
        assert float(delta_norm.half_step(kind, v)[-1]) == torch.finfo(kind).tiny * torch.finfo(kind).eps / 2


def test_chunks_of_states_that_grow():
    """Positive log decays among the others: the model by chunks is the rule there too."""
    a, rows = inputs((150, [0, 40, 150], 1, 2, 24, 16, F32, True, True))
    a["g"] = 0.3 * torch.randn(150, 2, generator=torch.Generator().manual_seed(1))
    want, got = ref.delta(**a)[0], delta_chunks.delta(**a)
    for name, w in want.items():
        assert float((got[name] - w).norm()) <= 1e-10 * float(w.norm()), name
