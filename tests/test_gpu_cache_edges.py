"""GPU: which keys a decode over 4-bit rows sums at lengths where one key is worth little, and the
gradients of norm and rotation against differences of the device's own forward."""
import numpy as np
import pytest

import gqa_inputs as gi
from tests import cache_edges as edges
from tests import cache_ref as ref
from tests.gpu_util import bits_of, from_dev, to_dev, torch_mod
from tests.test_gpu_cache import _dev, _dev_weights, _i32, _kv4_pools, _rope_inputs, _sync_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    torch_mod()
    import grouped_query_softmax_b200 as m
    return m


LONG = [
    # lengths, window, page, Hq, Hkv, D: one sequence in a cluster; many, in runs of tiles
    ([4099], 0, 64, 32, 8, 128), ([2000, 7000, 5121], 0, 16, 8, 2, 128), ([20001], 0, 128, 32, 2, 64), ([7000, 9000], 4096, 32, 8, 2, 128),
    ([7001, 4097] + [300 + i for i in range(150)], 0, 64, 8, 4, 128), ([20000] + [64 * i + 1 for i in range(120)], 0, 16, 16, 4, 64),
    ([9003, 5000] + [257 + i for i in range(150)], 2049, 32, 32, 2, 128),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: str((c[0][:3], len(c[0])) + c[1:]))
def test_decode_kv4_sums_each_key_once(gqa, case):
    lens, window, page, Hq, Hkv, D = case
    kp, vp, table = _kv4_pools(lens, Hkv, D, page, 131)
    q = gi.normal_bf16(132, gi.TENSOR_Q, (len(lens), Hq, 1, D))
    got = from_dev(gqa.attn_decode_kv4(to_dev(q), _dev(kp), _dev(vp), _i32(lens), _i32(table), window=window))
    _sync_ok(gqa)
    rng = np.random.default_rng(6)
    for b in list(range(3)) + [len(lens) - 1]:
        if b >= len(lens):
            continue
        n = lens[b]
        t = np.arange(n)
        at = table[b, t // page]
        lo = max(0, n - window) if window else 0
        keys = [lo, lo + 1, n - 1, n - 2, (lo // 64 + 1) * 64, (lo // 64 + 1) * 64 - 1, (n - 1) // 64 * 64, (n - 1) // 32 * 32 - 1]
        keys = sorted({int(j) for j in keys + list(rng.integers(lo, n, 6)) + ([lo - 1] if lo else []) if 0 <= j < n})
        o, off = edges.one_key_off(q[b, :, 0], kp[at, :, t % page], vp[at, :, t % page], lo, keys)
        edges.assert_sees(got[b, :, 0], o, off, f"sequence {b} of {n} keys")


@pytest.mark.parametrize("case", [(2, 64, 8, 2, 128, 128, False, True, True), (3, 50, 6, 2, 64, 32, True, True, False),
                                  (1, 40, 4, 4, 128, 64, False, False, False)], ids=str)
def test_norm_rope_gradients_match_differences_along_them(gqa, case):
    """<dz, f(up) - f(down)> = <gradient, up - down> for points either side of the inputs, in the direction
    of the gradient's signs, where it is largest: of q, of k and of the weights.

    Tolerance: outputs are off by at most 2^-8 of themselves, independently, with a deviation of at most
    2^-8 / sqrt(3): six deviations of their sum, and the gradient's the same; arithmetic in 32 bits 2^-15 of all terms; and what the
    formula's own difference, in 64 bits, is off by. It has to be under a twentieth of the gradient's part."""
    torch = torch_mod()
    B, T, Hq, Hkv, D, rot, inter, weighted, fp32 = case
    qkv, w, cos, sin, pos = _rope_inputs(case, 141)
    how = dict(_dev_weights(w, fp32), cos=_dev(cos), sin=_dev(sin), positions=_dev(pos), interleaved=inter, eps=1e-5)
    x = to_dev(qkv).transpose(1, 2)
    x = [x[:, :Hq].contiguous(), x[:, Hq:Hq + Hkv].contiguous()]
    dz = [to_dev(gi.normal_bf16(142 + i, gi.TENSOR_DO, tuple(x[i].shape))) for i in range(2)]
    grads = gqa.qk_norm_rope_bwd(*dz, *x, **how)
    c, s = cos[pos][:, None].astype(np.float64), sin[pos][:, None].astype(np.float64)
    f64 = lambda t: t.double().cpu().numpy()
    deviation = lambda *terms: 6 * 2.0 ** -8 / 3 ** 0.5 * np.sqrt(sum((t ** 2).sum() for t in terms))
    for i, name in enumerate(("q_weight", "k_weight")):
        d = f64(dz[i])
        for of in ("input", "weight") if weighted else ("input",):
            g = grads[i] if of == "input" else grads[2 + i]
            if of == "input":
                ends = [(x[i].float() + sign * g.float().sign() / 16).bfloat16() for sign in (1, -1)]
                z = [f64(gqa.qk_norm_rope(*((e, x[1]) if i == 0 else (x[0], e)), **how)[i]) for e in ends]
                exact = [ref.norm_rope(f64(e), w[name], 1e-5, c, s, inter)[0] for e in ends]
                ge = ref.norm_rope_bwd(d, f64(x[i]), w[name], 1e-5, c, s, inter)[0]
            else:  # linear in the weight: a step of 1 / 2 each way, exact in bf16 or not
                ends = [(how[name].float() + sign * g.sign() / 2).to(how[name].dtype) for sign in (1, -1)]
                z = [f64(gqa.qk_norm_rope(*x, **dict(how, **{name: e}))[i]) for e in ends]
                exact = [ref.norm_rope(f64(x[i]), f64(e), 1e-5, c, s, inter)[0] for e in ends]
                ge = ref.norm_rope_bwd(d, f64(x[i]), w[name], 1e-5, c, s, inter)[1]
            by = f64(ends[0]) - f64(ends[1])
            have, want = (d * (z[0] - z[1])).sum(), (f64(g) * by).sum()
            tol = abs((d * (exact[0] - exact[1])).sum() - (ge * by).sum())
            tol += deviation(d * z[0], d * z[1]) + (deviation(f64(g) * by) if of == "input" else 0)
            tol += 2.0 ** -15 * (np.abs(d * z[0]).sum() + np.abs(d * z[1]).sum())
            assert want > 0 and tol < want / 20, f"{of} of {name}: tolerance {tol:.3e} for {want:.3e}"
            assert abs(have - want) <= tol, f"{of} of {name}: {have:.6e} for {want:.6e}, tolerance {tol:.3e}"
    _sync_ok(gqa)


@pytest.mark.parametrize("B", [2, 120])
def test_decode_kv4_repeats_itself(gqa, B):
    """The same bits from call to call, whatever the workspace held before."""
    torch = torch_mod()
    lens = [(611 * i + 3000) % 5000 for i in range(B)]
    kp, vp, table = _kv4_pools(lens, 4, 64, 32, 151)
    q = to_dev(gi.normal_bf16(152, gi.TENSOR_Q, (B, 16, 2, 64)))
    args = (q, _dev(kp), _dev(vp), _i32(lens), _i32(table))
    need = gqa.gqa_attn_decode_kv4_workspace_bytes(B, 16, 4, 2, 5000, 64)
    assert (need > 0) == (B > 2)
    first = bits_of(gqa.attn_decode_kv4(*args, max_seqlen_k=5000))
    for byte in (0, 0x7F, 0xFF):
        ws = torch.full((max(need, 1),), byte, dtype=torch.uint8, device="cuda")
        again = gqa.attn_decode_kv4(*args, max_seqlen_k=5000, workspace=ws)
        _sync_ok(gqa)
        np.testing.assert_array_equal(bits_of(again), first)
