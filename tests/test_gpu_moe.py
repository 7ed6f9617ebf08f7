"""The mixture-of-experts layer for a few tokens against 64-bit arithmetic from its formula.

Tolerances, element by element, with u = 2^-23 (an ulp for each operation where a rounding
costs half of one).  A sum of D products: (D + 8) u sum |x w| =: e.  h = a(z) v with
|a'| <= 1.1 and a itself good to 8 u (a ReLU's zero may stand on either side of a z within e_z):
|dh| <= 1.1 e_z |v| + (|a| + 1.1 e_z) e_v + 9 u |h|.  y: the slots' weights (wrong by at most (E + 40) u of
themselves, and by |w| (|dl| + |dl'|) for logits that are e_l off), the sum over F neurons, k slots and
the parts an expert is split into:
  sum w (sum |dh| |Wd| + (F + 64) u sum |h Wd|) + sum |dw| |sum h Wd|
A bf16 y: half a bf16 step, 2^-8 of it, more.  A choice is compared where its logits are further
apart than 2 e_l.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gated_gate_gb300 as tw
from tests._gpu import ensure_built

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def f64(t):
    return t.double().cpu().numpy()


def values(w):
    if not isinstance(w, tw.Int4):
        return f64(w)
    j = torch.arange(w.K, device=w.code.device) // w.group
    z = 8.0 if w.zero is None else w.zero.double()[..., j]
    return f64((w.codes().double() - z) * w.scale.double()[..., j])


def layer(E, F, D, bits, seed=0, density=0.5, group=64, zero_points=True, router=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    shift = 1.6 * float(torch.erfinv(torch.tensor(2 * density - 1))) / D ** 0.5
    w = [torch.randn((E, F, D), generator=g) / D ** 0.5 for _ in range(3)]
    w[0] += shift / (0.5 * D ** 0.5)
    r = (2 * torch.randn((E, D), generator=g) / D ** 0.5).to(router).cuda()
    if bits == 4:
        return r, [tw.twell_quant_int4(v.cuda(), group=group, zero_points=zero_points) for v in w]
    return r, [v.to(torch.bfloat16).cuda() for v in w]


def tokens(T, D, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, D), generator=g) + 0.5).to(torch.bfloat16).cuda()


def act64(z, act):
    if act == "relu":
        return np.where(z <= 0, 0.0, z)
    with np.errstate(over="ignore"):
        return z / (1 + np.exp(-z))


def check_y(o, x, w, act, weights64, dw):
    """y against the choice that the call made: weights64 [T][k] and their error dw."""
    x, (wg, wu, wd) = f64(x), (values(v) for v in w)
    ids = o.ids.cpu().numpy()
    E, F, D = wg.shape
    T, k = ids.shape
    ref, tol = np.zeros((T, D)), np.zeros((T, D))
    for e in range(E):
        t, s = np.nonzero(ids == e)
        if not len(t):
            continue
        xe, c = x[t], (D + 8) * U
        z, v = xe @ wg[e].T, xe @ wu[e].T
        ez, ev = c * np.abs(xe) @ np.abs(wg[e]).T, c * np.abs(xe) @ np.abs(wu[e]).T
        a = act64(z, act)
        h = a * v
        dh = 1.1 * ez * np.abs(v) + (np.abs(a) + 1.1 * ez) * ev + 9 * U * np.abs(h)
        y, p = h @ wd[e], np.abs(weights64[t, s])[:, None]
        err = p * (dh @ np.abs(wd[e]) + (F + 64) * U * (np.abs(h) @ np.abs(wd[e])))
        np.add.at(ref, t, weights64[t, s][:, None] * y)
        np.add.at(tol, t, err + dw[t, s][:, None] * np.abs(y))
    if o.y.dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    got = f64(o.y)
    assert got.shape == ref.shape
    bad = np.abs(got - ref) - tol
    assert (bad <= 0).all(), (np.unravel_index(bad.argmax(), bad.shape), bad.max())


def check_choice(o, x, r, k, renormalise):
    """The choice against 64-bit logits; returns its weights in 64 bits and their error."""
    xd, rd = f64(x), f64(r)
    E, D = rd.shape
    logits = xd @ rd.T
    e = (D + 8) * U * (np.abs(xd) @ np.abs(rd).T)
    ids = o.ids.cpu().numpy().astype(np.int64)
    order = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    T = len(ids)
    row = np.arange(T)[:, None]
    assert ((0 <= ids) & (ids < E)).all() and all(len(set(i)) == k for i in ids.tolist())
    # in the place of each chosen expert stands one whose logit is as large, to rounding
    off = np.abs(logits[row, ids] - logits[row, order])
    assert (off <= e[row, ids] + e[row, order]).all()
    top = logits.max(1, keepdims=True)
    p = np.exp(logits - top)
    w = p[row, ids] / (p[row, ids] if renormalise else p).sum(1, keepdims=True)
    dw = w * ((E + 40) * U + 2.2 * e.max(1, keepdims=True))
    assert (np.abs(f64(o.weights) - w) <= dw).all()
    return w, dw


@pytest.mark.parametrize("bits,group,zero_points", [(16, 0, False), (4, 32, False), (4, 32, True),
                                                    (4, 64, True), (4, 128, False)])
@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("T,E,k,F,D", [
    (1, 1, 1, 1, 8), (1, 4, 2, 16, 64), (1, 64, 8, 100, 256), (2, 5, 5, 33, 136),
    (3, 33, 4, 300, 1000), (8, 16, 3, 64, 1536), (9, 8, 2, 40, 520), (16, 3, 1, 130, 200),
    (40, 6, 4, 50, 72), (64, 64, 8, 48, 128), (70, 2, 1, 20, 640)])
def test_layer(T, E, k, F, D, act, bits, group, zero_points):
    r, w = layer(E, F, D, bits, seed=T, group=group, zero_points=zero_points)
    x = tokens(T, D)
    for renormalise, dtype in ((True, torch.float32), (False, torch.bfloat16)):
        o = tw.twell_moe_decode(x, r, *w, top_k=k, act=act, renormalise=renormalise, dtype=dtype)
        wt, dw = check_choice(o, x, r, k, renormalise)
        check_y(o, x, w, act, wt, dw)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("T,E,k,F,D,density", [(1, 8, 2, 1000, 2048, 0.01), (5, 4, 2, 500, 512, 0.03),
                                               (20, 8, 3, 260, 384, 0.005), (1, 2, 1, 64, 64, 0.0005)])
def test_sparse_gates(T, E, k, F, D, density, bits):
    """Few gates are positive: neurons, rounds and whole parts without one."""
    r, w = layer(E, F, D, bits, seed=3, density=density, group=128, zero_points=False)
    x = tokens(T, D)
    o = tw.twell_moe_decode(x, r, *w, top_k=k)
    wt, dw = check_choice(o, x, r, k, True)
    check_y(o, x, w, "relu", wt, dw)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("act,density", [("relu", 0.5), ("relu", 0.03), ("silu", 0.5)])
@pytest.mark.parametrize("T,E,k", [(8, 32, 8), (64, 16, 2)])
def test_many_neurons(T, E, k, act, density, bits):
    """More than a round of neurons a block: tiles whose columns several warps divide unevenly,
    slabs that begin within a block's share, chunks of h."""
    F, D = 2100, 520
    r, w = layer(E, F, D, bits, seed=12, density=density, group=64)
    x = tokens(T, D)
    o = tw.twell_moe_decode(x, r, *w, top_k=k, act=act)
    wt, dw = check_choice(o, x, r, k, True)
    check_y(o, x, w, act, wt, dw)


@pytest.mark.parametrize("bits,T,D", [(16, 2, 16384), (4, 12, 8200), (16, 12, 8192), (4, 1, 9000)])
def test_wide(bits, T, D):
    r, w = layer(3, 24, D, bits, seed=5, group=32)
    x = tokens(T, D)
    o = tw.twell_moe_decode(x, r, *w, top_k=2, act="silu")
    wt, dw = check_choice(o, x, r, 2, True)
    check_y(o, x, w, "silu", wt, dw)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("T,E,k", [(1, 3, 2), (13, 10, 3), (6, 4, 8), (50, 2, 4), (256, 4, 8)])
def test_routed(T, E, k, bits):
    """The caller's choice: absent experts, the same one twice, tokens without any, weights of
    any sign, an expert with more pairs than are taken at a time."""
    F, D = 70, 264
    _, w = layer(E, F, D, bits, seed=7)
    x = tokens(T, D)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, dtype=torch.int32)
    ids[ids == E] = 2 ** 31 - 1
    ids[T // 2] = -5
    if T > 2:
        ids[2] = 1
    weights = torch.randn((T, k), generator=g)
    given = ids.clone()
    weights[(ids < 0) | (ids >= E)] = float("nan")   # of no expert: not used
    ids, weights = ids.cuda(), weights.cuda()
    for act in ("relu", "silu"):
        o = tw.twell_moe_decode(x, None, *w, act=act, ids=ids, weights=weights)
        assert torch.equal(ids.cpu(), given)
        check_y(o, x, w, act, np.nan_to_num(f64(weights)), np.zeros((T, k)))
        none = ((given < 0) | (given >= E)).all(1)
        assert none.any() and not o.y[none.cuda()].any()


def test_nobody_routed():
    _, w = layer(3, 40, 128, 16)
    x = tokens(5, 128)
    ids = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    y = torch.full((5, 128), 3.0, device="cuda")
    tw.twell_moe_decode(x, None, *w, ids=ids, weights=torch.ones((5, 2), device="cuda"), y=y)
    assert not y.any()


@pytest.mark.parametrize("E", [8, 40])
def test_ties(E):
    """Equal rows of the router: the lowest experts, in order."""
    _, w = layer(E, 16, 64, 16)
    r = torch.randn((1, 64)).expand(E, 64).contiguous().to(torch.bfloat16).cuda()
    r[3] = -r[3]
    for T in (1, 9):
        x = tokens(T, 64)
        o = tw.twell_moe_decode(x, r, *w, top_k=4)
        up = (f64(x) @ f64(r[0])) > 0
        for t in range(T):
            assert o.ids[t].tolist() == ([0, 1, 2, 4] if up[t] else [3, 0, 1, 2])
    zero = torch.zeros_like(r)
    zero[5] = -0.0
    o = tw.twell_moe_decode(tokens(2, 64), zero, *w, top_k=8)
    assert o.ids.tolist() == [list(range(8))] * 2
    assert torch.equal(o.weights, torch.full((2, 8), 0.125, device="cuda"))


@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("bits", [4, 16])
def test_not_finite(bits, act, T):
    """A token's NaN stays in the token, an expert's with its tokens; what a neuron whose
    gate is not positive holds elsewhere is not used.  (The other tokens' sums may be taken
    in another order, by the experts and neurons that are active: they are held against
    the formula, not against the bits of another call.)"""
    E, F, D, k = 6, 40, 256, 2
    r, w = layer(E, F, D, bits, seed=2)
    x = tokens(T, D)
    ref = tw.twell_moe_decode(x, r, *w, top_k=k, act=act)
    bad = x.clone()
    bad[1, 7] = float("nan")
    o = tw.twell_moe_decode(bad, r, *w, top_k=k, act=act)


    def others_stand(o, rows):
        some = tw.Moe(o.y[rows], o.ids[rows], o.weights[rows])
        check_y(some, x[rows], w, act, *check_choice(some, x[rows], r, k, True))

    keep = torch.arange(T, device="cuda") != 1
    assert o.y[1].isnan().all() and o.weights[1].isnan().all()
    assert torch.equal(o.ids[1].cpu(), torch.arange(k, dtype=torch.int32))
    others_stand(o, keep)
    e = int(ref.ids[0, 0])
    dead = [v.clone() if bits == 16 else tw.Int4(v.code.clone(), v.scale.clone(), v.zero.clone(),
                                                 v.K, v.group) for v in w]
    (dead[1] if bits == 16 else dead[1].scale)[e] = float("nan")
    o = tw.twell_moe_decode(x, r, *dead, top_k=k, act=act)
    hit = (ref.ids == e).any(1)
    assert o.y[hit].isnan().all()
    others_stand(o, ~hit)
    if act == "relu":
        (dead[0] if bits == 16 else dead[0].scale)[e] = 0.0
        o = tw.twell_moe_decode(x, r, *dead, top_k=k, act=act)
        assert not o.y.isnan().any()
        others_stand(o, ~hit)
    inf = r.clone()
    inf[0] = float("inf")
    o = tw.twell_moe_decode(x.abs(), inf, *w, top_k=k, act=act)
    assert (o.ids[:, 0] == 0).all() and o.weights.isnan().all()


def test_repeats_outputs_streams():
    r, w = layer(16, 200, 512, 4, seed=4)
    x = tokens(24, 512)
    ref = tw.twell_moe_decode(x, r, *w, top_k=4)
    ws = torch.full((tw.twell_moe_decode_workspace(24, 512, 200, 16, 4),), 255, dtype=torch.uint8,
                    device="cuda")
    y = torch.empty((24, 512), device="cuda")
    for _ in range(4):
        y.fill_(7.0)
        o = tw.twell_moe_decode(x, r, *w, top_k=4, y=y, ws=ws, ids=ref.ids.clone(),
                                weights=torch.zeros_like(ref.weights))
        assert o.y is y and torch.equal(y, ref.y)
        assert torch.equal(o.ids, ref.ids) and torch.equal(o.weights, ref.weights)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):   # calls at once, each with a workspace of its own
        got += [tw.twell_moe_decode(x, r, *w, top_k=4, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o.y, ref.y) for o in got)
    o = tw.twell_moe_decode(x, None, *w, ids=ref.ids, weights=ref.weights)
    assert torch.equal(o.y, ref.y)


def test_graph():
    r, w = layer(32, 96, 256, 16, seed=4)
    x = tokens(4, 256)
    tw.twell_moe_decode(x, r, *w, top_k=4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = tw.twell_moe_decode(x, r, *w, top_k=4)
        b = tw.twell_moe_decode(a.y.to(torch.bfloat16), r, *w, top_k=4)
    for seed in (5, 6, 7):
        x.copy_(tokens(4, 256, seed))
        graph.replay()
        ra = tw.twell_moe_decode(x, r, *w, top_k=4)
        rb = tw.twell_moe_decode(ra.y.to(torch.bfloat16), r, *w, top_k=4)
        assert torch.equal(a.y, ra.y) and torch.equal(b.y, rb.y) and torch.equal(b.ids, rb.ids)


def test_one_ffn_is_one_expert():
    """E = 1: a gated FFN of 4-bit weights for a decode batch."""
    _, w = layer(1, 600, 1024, 4, seed=9, density=0.02, group=128)
    x = tokens(7, 1024)
    ids = torch.zeros((7, 1), dtype=torch.int32, device="cuda")
    o = tw.twell_moe_decode(x, None, *w, ids=ids, weights=torch.ones((7, 1), device="cuda"))
    check_y(o, x, w, "relu", np.ones((7, 1)), np.zeros((7, 1)))


def test_no_tokens():
    r, w = layer(4, 16, 64, 16)
    o = tw.twell_moe_decode(tokens(0, 64), r, *w, top_k=2)
    assert o.y.shape == (0, 64) and o.ids.shape == (0, 2)


def test_workspace_of_the_largest_batch():
    """One workspace for a loop whose batch shrinks, though fewer tokens are divided into more
    parts: 15 tokens and one expert are one slab in 8 parts, 16 may be two slabs in 4."""
    D, F, E, k = 2048, 1200, 1, 1
    sizes = [tw.twell_moe_decode_workspace(T, D, F, E, k) for T in range(41)]
    assert sizes == sorted(sizes) and sizes[1] > 0
    ws = torch.full((sizes[16],), 255, dtype=torch.uint8, device="cuda")
    r, w = layer(E, F, D, 16, seed=2)
    x = tokens(16, D)
    for T in (16, 15, 9, 8, 1, 0):
        o = tw.twell_moe_decode(x[:T], r, *w, top_k=k, ws=ws)
        assert torch.equal(o.y, tw.twell_moe_decode(x[:T], r, *w, top_k=k).y)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (8, 64, 8), (8, 3, 3), (9, 200, 1), (64, 16, 2),
                                   (256, 30, 8), (256, 500, 8)])
def test_stays_within_its_workspace(T, E, k, bits):
    D, F = 136, 50
    r, w = layer(E, F, D, bits, seed=6, group=32)
    x = tokens(T, D)
    need = tw.twell_moe_decode_workspace(T, D, F, E, k)
    buf = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    for act in ("relu", "silu"):
        o = tw.twell_moe_decode(x, r, *w, top_k=k, act=act, ws=buf[:need])
        assert torch.equal(o.y, tw.twell_moe_decode(x, r, *w, top_k=k, act=act).y)
    one = torch.zeros((T, k), dtype=torch.int32, device="cuda")   # all with one expert
    tw.twell_moe_decode(x, None, *w, ids=one, weights=o.weights, ws=buf[:need])
    assert (buf[need:] == 171).all()


# ------------------------------------------- refusals of the binding


def test_refusals():
    r, w = layer(4, 32, 64, 16)
    x = tokens(3, 64)
    four = [tw.twell_quant_int4(v, group=32) for v in w]
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    weights = torch.ones((3, 2), device="cuda")

    def bad(error, *a, **k):
        with pytest.raises(error):
            tw.twell_moe_decode(*a, **k)

    bad(TypeError, x.float(), r, *w, top_k=2)
    bad(ValueError, x[:, :32], r, *w, top_k=2)
    bad(ValueError, tokens(6, 64)[::2], r, *w, top_k=2)
    bad(ValueError, x, r, *w)
    bad(ValueError, x, r, *w, top_k=2, act="gelu")
    bad(ValueError, x, r[:3], *w, top_k=2)
    bad(TypeError, x, r.half(), *w, top_k=2)
    bad(TypeError, x, r.cpu(), *w, top_k=2)
    bad(ValueError, x, r, w[0], w[1], w[2][:3], top_k=2)
    bad(TypeError, x, r, w[0], w[1], w[2].float(), top_k=2)
    bad(TypeError, x, r, w[0][0], w[1], w[2], top_k=2)
    bad(TypeError, x, r, four[0], w[1], four[2], top_k=2)
    bad(TypeError, x, r, w[0], four[1], w[2], top_k=2)
    bad(ValueError, x, r, four[0], four[1], tw.twell_quant_int4(w[2], group=64), top_k=2)
    bad(ValueError, x, r, four[0], four[1], tw.twell_quant_int4(w[2][:, :16].contiguous(),
                                                                 group=32), top_k=2)
    bad(ValueError, x, None, *w, ids=ids)
    bad(ValueError, x, None, *w, weights=weights)
    bad(TypeError, x, None, *w, ids=ids.long(), weights=weights)
    bad(ValueError, x, None, *w, ids=ids[:2], weights=weights)
    bad(ValueError, x, None, *w, ids=ids, weights=weights[:, :1])
    bad(ValueError, x, r, *w, top_k=2, ids=ids[:, :1].contiguous())
    bad(TypeError, x, r, *w, top_k=2, dtype=torch.float16)
    bad(ValueError, x, r, *w, top_k=2, y=torch.empty((3, 32), device="cuda"))
    bad(TypeError, x, r, *w, top_k=2, ws=torch.empty((1 << 20,)))
    bad(tw.TwellError, x, r, *w, top_k=2, ws=torch.empty((64,), dtype=torch.uint8, device="cuda"))
    bad(tw.TwellError, x, r, *w, top_k=5)
    many = tokens(257, 64)
    bad(tw.TwellError, many, r, *w, top_k=2)
    odd = layer(2, 8, 60, 16)
    bad(tw.TwellError, tokens(2, 60), odd[0], *odd[1], top_k=1)
    held = torch.empty((4 * 32 * 64 + 4,), dtype=torch.bfloat16, device="cuda")
    off = held[4:].view(4, 32, 64)   # rows off 16-byte boundaries
    bad(tw.TwellError, x, r, off, w[1], w[2], top_k=2)
    y = tw.twell_moe_decode(x, r, *w, top_k=2).y
    assert y.isfinite().all()        # the context is as it was


def test_more_than_2_31_elements():
    """Experts behind 2^31 elements, in both forms."""
    E, F, D = 36, 15000, 4096
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    x = tokens(3, D)
    w = [torch.zeros((E, F, D), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    g = torch.Generator(device="cuda").manual_seed(1)
    last = [torch.randn((F, D), generator=g, device="cuda") / D ** 0.5 for _ in range(3)]
    for a, b in zip(w, last):
        a[E - 1] = b
    ids = torch.full((3, 1), E - 1, dtype=torch.int32, device="cuda")
    one = torch.zeros_like(ids)
    weights = torch.ones((3, 1), device="cuda")
    small = [v[E - 1:].contiguous() for v in w]
    # (a single expert's products are divided as one of many are: the same bits)
    y = tw.twell_moe_decode(x, None, *w, ids=ids, weights=weights).y
    ref = tw.twell_moe_decode(x, None, *small, ids=one, weights=weights)
    assert y.any() and torch.allclose(y, ref.y, rtol=1e-5, atol=1e-5 * float(ref.y.abs().max()))
    four = []
    for i in range(3):
        four.append(tw.twell_quant_int4(w[i]))
        w[i] = None
    y = tw.twell_moe_decode(x, None, *four, ids=ids, weights=weights).y
    small = [tw.Int4(q.code[E - 1:].clone(), q.scale[E - 1:].clone(), None, D, 128) for q in four]
    ref = tw.twell_moe_decode(x, None, *small, ids=one, weights=weights)
    assert y.any() and torch.allclose(y, ref.y, rtol=1e-5, atol=1e-5 * float(ref.y.abs().max()))
