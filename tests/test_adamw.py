"""adamw_step: the update and the moments against float64, the stochastic
rounding against its definition, many ragged and unaligned tensors, streams and
graphs, and the refusals of the C entry point and of the binding."""
import ctypes
import os
import random

import numpy as np
import pytest
import torch

import quantized_collective_payloads_amd as qcp
from tests import operator_reference as R

GPU = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
# rounding unit of fp32; the bounds below count the roundings of each formula
U = 2.0 ** -24


@pytest.fixture()
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    qcp.library()


def flat_views(sizes, dtype, gap, seed, sigma):
    """Tensors of `sizes` as views of one buffer, `gap` elements apart: odd gaps
    and sizes leave them aligned to their element only."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    buf = (torch.randn(sum(sizes) + gap * (len(sizes) + 1), generator=g, device="cuda") * sigma).to(dtype)
    out, at = [], gap
    for n in sizes:
        out.append(buf[at:at + n])
        at += n + gap
    return out, buf


def host(ts):
    return [t.detach().to(torch.float64).cpu().numpy() for t in ts]


def check_update(p_new, p_old, g, m, v, step, h, scale, what):
    """p against float64: the two products and the subtraction round p once each,
    the update takes about ten roundings and a reciprocal good to 1 ulp."""
    want, _, _ = R.adamw(p_old, g, m, v, step, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"], scale)
    up = np.abs(want - p_old * (1 - h["lr"] * h["weight_decay"]))
    # the update's own cancellation: m is a sum of two terms rounded on its own
    parts = h["beta1"] * np.abs(m) + (1 - h["beta1"]) * np.abs(g * scale)
    top = np.abs(R.adamw(p_old, g, m, v, step, h["lr"], h["beta1"], h["beta2"], h["eps"], 0.0, scale)[1])
    wide = up * np.where(top > 0, parts / np.maximum(top, 1e-300), 1.0)
    bound = 4 * U * np.abs(p_old) + 24 * U * (up + wide) + 1e-37
    bad = np.nonzero(~(np.abs(p_new - want) <= bound))[0]
    assert bad.size == 0, (what, bad[:4], p_new[bad[:4]], want[bad[:4]])


SIZES = [
    [1], [3], [4], [5], [31, 32, 33], [1024], [4096], [4097], [1, 2, 3, 4, 5, 6, 7, 1023, 1025],
    [4095, 1, 8191, 130], [20_001],
]


@GPU
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("gt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ct", [None, "f16", "bf16"])
def test_fp32_moments(gpu, sizes, gt, ct):
    G = 64
    params, _ = flat_views(sizes, torch.float32, 3, 1, 0.02)
    copies = None if ct is None else flat_views(sizes, DT[ct], 1, 2, 1.0)[0]
    opt = qcp.AdamW(params, copies=copies, state="f32", G=G)
    scale = torch.tensor([0.37], device="cuda")
    for step in (1, 2, 3):
        grads, _ = flat_views(sizes, DT[gt], 5, 10 + step, 1e-3)
        p0, g = host(params), host(grads)
        m0, v0 = host([opt.m])[0], host([opt.v])[0]
        qcp.adamw_step(opt, grads, step, grad_scale=scale, **HYPER)
        m1, v1 = host([opt.m])[0], host([opt.v])[0]
        p1 = host(params)
        for i, n in enumerate(sizes):
            at = slice(opt.offsets[i], opt.offsets[i] + n)
            s = float(np.float32(0.37))
            _, m, v = R.adamw(p0[i], g[i], m0[at], v0[at], step, HYPER["lr"], 0.9, 0.999, 1e-8, 0.1, s)
            parts = 0.9 * np.abs(m0[at]) + 0.1 * np.abs(g[i]) * s
            assert (np.abs(m1[at] - m) <= 5 * U * parts + 1e-44).all()      # 4 roundings, 2 constants
            assert (np.abs(v1[at] - v) <= 8 * U * v + 1e-44).all()          # 5 roundings, 2 constants
            check_update(p1[i], p0[i], g[i], m0[at], v0[at], step, HYPER, s, (sizes, gt, step, i))
            if copies is not None:
                assert torch.equal(copies[i], params[i].to(DT[ct]))
            pad = slice(opt.offsets[i] + n, opt.offsets[i] + qcp.n_blocks(n, G) * G)
            assert not m1[pad].any() and not v1[pad].any()


def check_eight(opt, sizes, p0, g, old, step, seed, h, scale, p1):
    """The 8-bit moments after a step: each tensor's scales and codes, from the
    moments `old` decoded before it."""
    mv0, rv0 = old
    G = opt.G
    ms, vs = host([opt.m_scales])[0], host([opt.v_scales])[0]
    mc, vc = opt.m.cpu().numpy(), opt.v.cpu().numpy()
    for i, n in enumerate(sizes):
        o, N = opt.offsets[i], qcp.n_blocks(n, G) * G
        m0, r0 = mv0[o:o + n], rv0[o:o + n]
        _, m, v = R.adamw(p0[i], g[i], m0, r0 * r0, step, h["lr"], h["beta1"], h["beta2"], h["eps"], 0.0, scale)
        check_update(p1[i], p0[i], g[i], m0, r0 * r0, step, h, scale, (sizes, step, i))
        low, high = R.random_halves(np.arange(o, o + N), seed, step)
        for x, codes, scales, half, least in ((m, mc, ms, low, False), (np.sqrt(v), vc, vs, high, True)):
            x = np.pad(x, (0, N - n))
            s = scales[o // G:(o + N) // G]
            want = R.block_scale(x, G)
            near = R.block_scale(x * (1 + 16 * U), G)      # an absmax at 448 * 2^k may round either way
            under = R.block_scale(x * (1 - 16 * U), G)
            assert ((s == want) | (s == near) | (s == under)).all()
            s = np.repeat(s, G)
            got = R.e4m3_value(codes[o:o + N])
            # x / spacing is off by at most 16 * 8 rounding units, so only a value that
            # close to its random threshold may go the other way; m's two terms may cancel
            parts = np.abs(x) if least else np.pad(h["beta1"] * np.abs(m0) + (1 - h["beta1"]) * np.abs(g[i] * scale), (0, N - n))
            slack = 256 * U * np.where(x != 0, parts / np.maximum(np.abs(x), 1e-300), 1.0) + 2.0 ** -19
            a, b = R.stochastic_e4m3(x, s, half, -slack), R.stochastic_e4m3(x, s, half, slack)
            if least:
                a, b = np.where(x > 0, np.maximum(a, 2.0 ** -9), 0), np.where(x > 0, np.maximum(b, 2.0 ** -9), 0)
            bad = np.nonzero(~((got >= np.minimum(a, b)) & (got <= np.maximum(a, b))))[0]
            assert bad.size == 0, (sizes, step, i, least, bad[:4], got[bad[:4]], a[bad[:4]], b[bad[:4]])
            assert not codes[o + n:o + N].any()


def decoded(opt):
    return (R.e4m3_value(opt.m.cpu().numpy()) * np.repeat(host([opt.m_scales])[0], opt.G),
            R.e4m3_value(opt.v.cpu().numpy()) * np.repeat(host([opt.v_scales])[0], opt.G))


@GPU
@pytest.mark.parametrize("G", [32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("gt", ["f32", "bf16", "f16"])
def test_e4m3_moments(gpu, sizes, G, gt):
    params, _ = flat_views(sizes, torch.float32, 1, 3, 0.02)
    copies, _ = flat_views(sizes, torch.bfloat16, 3, 4, 1.0)
    opt = qcp.AdamW(params, copies=copies, state="e4m3", G=G)
    for step in (1, 2, 3):
        grads, _ = flat_views(sizes, DT[gt], 1, 20 + step, 1e-3 * 10 ** step)
        if step == 2:
            for g in grads:
                g[::3] = 0                                # some moments only decay
        p0, g, old = host(params), host(grads), decoded(opt)
        qcp.adamw_step(opt, grads, step, seed=5, **HYPER)
        check_eight(opt, sizes, p0, g, old, step, 5, HYPER, 1.0, host(params))
        for c, p in zip(copies, params):
            assert torch.equal(c, p.to(torch.bfloat16))


@GPU
def test_many_tensors_over_several_launches(gpu):
    """150 tensors are three launches; empty ones take none."""
    r = random.Random(4)
    sizes = [0 if i % 17 == 5 else r.choice((1, 2, 3, 7, 100, 129, 4096, 5000, 9001)) for i in range(150)]
    params, _ = flat_views(sizes, torch.float32, 1, 5, 0.02)
    grads, _ = flat_views(sizes, torch.bfloat16, 1, 6, 1e-3)
    opt = qcp.AdamW(params, state="e4m3", G=128)
    p0, g, old = host(params), host(grads), decoded(opt)
    qcp.adamw_step(opt, grads, 1, seed=9, **HYPER)
    check_eight(opt, sizes, p0, g, old, 1, 9, HYPER, 1.0, host(params))


@GPU
def test_more_tensors_than_a_call_takes(gpu):
    sizes = [1 + i % 37 for i in range(2100)]
    params, _ = flat_views(sizes, torch.float32, 1, 5, 0.02)
    grads, _ = flat_views(sizes, torch.float32, 1, 6, 1e-3)
    copies, _ = flat_views(sizes, torch.float16, 1, 7, 1.0)
    opt = qcp.AdamW(params, copies=copies, state="e4m3", G=32)
    p0, g, old = host(params), host(grads), decoded(opt)
    qcp.adamw_step(opt, grads, 1, seed=9, **HYPER)
    check_eight(opt, sizes, p0, g, old, 1, 9, HYPER, 1.0, host(params))
    assert all(torch.equal(c, p.to(torch.float16)) for c, p in zip(copies, params))


@GPU
def test_nothing_outside_the_tensors_is_written(gpu):
    sizes = [5, 1, 4099, 64, 3]
    params, pbuf = flat_views(sizes, torch.float32, 7, 7, 0.02)
    copies, cbuf = flat_views(sizes, torch.float16, 7, 8, 1.0)
    grads, _ = flat_views(sizes, torch.float32, 7, 9, 1e-3)
    p0, c0 = pbuf.clone(), cbuf.clone()
    inside = torch.zeros(pbuf.numel(), dtype=torch.bool, device="cuda")
    at = 7
    for n in sizes:
        inside[at:at + n] = True
        at += n + 7
    opt = qcp.AdamW(params, copies=copies, state="e4m3", G=32)
    tail = torch.full((opt.n_state + 512,), 0x55, dtype=torch.uint8, device="cuda")
    tail[:opt.n_state] = 0
    opt = qcp.AdamW(params, copies=copies, state="e4m3", G=32, m=tail)
    qcp.adamw_step(opt, grads, 1, **HYPER)
    assert torch.equal(pbuf[~inside], p0[~inside]) and torch.equal(cbuf[~inside], c0[~inside])
    assert not torch.equal(pbuf[inside], p0[inside])
    assert (tail[opt.n_state:] == 0x55).all()


@GPU
def test_extreme_gradients(gpu):
    """Zero gradients leave a zero state; tiny and huge ones stay finite; a
    positive second moment never becomes zero beside a huge neighbour."""
    n = 2048
    p = torch.zeros(n, device="cuda")
    opt = qcp.AdamW([p], state="e4m3", G=128)
    qcp.adamw_step(opt, [torch.zeros(n, device="cuda")], 1, **HYPER)
    assert not p.any() and not opt.m.any() and not opt.v.any() and not opt.m_scales.any()
    g = torch.full((n,), 1e-12, device="cuda")
    g[::128] = 1e4
    g[1::128] = -1e-18
    qcp.adamw_step(opt, [g], 2, **HYPER)
    assert torch.isfinite(p).all()
    r = R.e4m3_value(opt.v.cpu().numpy())
    assert (r > 0).all()                                  # 1e-18 beside 1e4 in one block
    qcp.adamw_step(opt, [torch.zeros(n, device="cuda")], 3, **HYPER)
    assert torch.isfinite(p).all()


@GPU
def test_stochastic_rounding_is_unbiased_where_nearest_would_freeze(gpu):
    """A second moment that decays by 1/1000 a step: over 2000 steps of zero
    gradients its mean follows 0.999^t (rounding to nearest would leave every code
    where it is).  Mean of 65,536 values: standard error below 1%."""
    n = 65536
    p = torch.zeros(n, device="cuda")
    opt = qcp.AdamW([p], state="e4m3", G=128)
    g = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") + 0.5
    g[::128] = 2.0
    qcp.adamw_step(opt, [g], 1, seed=1, **HYPER)
    first = decoded(opt)[1]
    zero = torch.zeros(n, device="cuda")
    steps = 500
    for t in range(2, 2 + steps):
        qcp.adamw_step(opt, [zero], t, seed=1, **HYPER)
    ratio = decoded(opt)[1].mean() / first.mean()
    assert abs(ratio / 0.999 ** (steps / 2) - 1) < 0.02, ratio


@GPU
def test_same_seed_same_bytes_other_seed_other_bytes(gpu):
    sizes = [70_001, 513]
    grads, _ = flat_views(sizes, torch.float32, 0, 1, 1e-3)

    def once(seed):
        params, _ = flat_views(sizes, torch.float32, 0, 2, 0.02)
        opt = qcp.AdamW(params, state="e4m3", G=128)
        for step in (1, 2):
            qcp.adamw_step(opt, grads, step, seed=seed, **HYPER)
        return opt
    a, b, c = once(1 << 40), once(1 << 40), once(2 << 40)
    assert torch.equal(a.m, b.m) and torch.equal(a.v, b.v)
    assert not torch.equal(a.m, c.m) and not torch.equal(a.v, c.v)


@GPU
def test_side_stream_and_graph(gpu):
    """On a side stream, and captured: a graph's replays each equal an eager step
    with the same arguments, with eager work in between; the clipping factor is
    read on the device, so a replay takes the value it then has."""
    sizes = [3000, 1, 4097]
    grads, _ = flat_views(sizes, torch.bfloat16, 0, 1, 1e-3)
    scale = torch.ones(1, device="cuda")

    def make():
        params, _ = flat_views(sizes, torch.float32, 0, 2, 0.02)
        return qcp.AdamW(params, state="e4m3", G=64)

    def state(o):
        return [t.clone() for t in (*o.params, o.m, o.v, o.m_scales, o.v_scales)]
    eager, want = make(), []
    for k in range(4):
        scale.fill_(1.0 / (k + 1))
        qcp.adamw_step(eager, grads, 7, grad_scale=scale, seed=3, **HYPER)
        want.append(state(eager))
    replayed = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        warm = make()
        qcp.adamw_step(warm, grads, 7, grad_scale=scale, seed=3, **HYPER)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qcp.adamw_step(replayed, grads, 7, grad_scale=scale, seed=3, **HYPER)
    for k in range(4):
        scale.fill_(1.0 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(state(replayed), want[k]):
            assert torch.equal(a, b), k


@GPU
def test_moments_past_32_bits(gpu):
    """A tensor whose moments begin beyond element 2^32 (the codes of one flat
    8-bit buffer): places, scales and the hash's high word."""
    G, first = 128, (1 << 32) + 256
    n = 1000
    m = torch.zeros(first + 1024, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(m)
    ms, vs = (torch.zeros(m.numel() // G, device="cuda") for _ in range(2))
    p = torch.randn(n, device="cuda") * 0.02
    g = torch.randn(n, device="cuda") * 1e-3
    p0 = host([p])[0]
    arr = lambda t, x: (t * 1)(x)  # noqa: E731
    rc = qcp.library().adamw_step(
        arr(ctypes.c_void_p, p.data_ptr()), arr(ctypes.c_void_p, g.data_ptr()), None,
        arr(ctypes.c_int64, n), arr(ctypes.c_int64, first), 1, 3, 0, 0x43, m.data_ptr(), ms.data_ptr(),
        v.data_ptr(), vs.data_ptr(), m.numel(), G, 1, 3e-4, 0.9, 0.999, 1e-8, 0.1, None, 11, None)
    assert rc == 0
    torch.cuda.synchronize()
    assert not m[:first].any() and not ms[:first // G].any()

    class View:
        pass
    o = View()
    o.G, o.offsets = G, [0]
    _, mm, vv = R.adamw(p0, host([g])[0], 0 * p0, 0 * p0, 1, 3e-4, 0.9, 0.999, 1e-8, 0.1)
    low, high = R.random_halves(np.arange(first, first + n), 11, 1)
    for x, codes, scales, half in ((mm, m, ms, low), (np.sqrt(vv), v, vs, high)):
        s = np.repeat(host([scales[first // G:]])[0], G)[:n]
        got = R.e4m3_value(codes[first:first + n].cpu().numpy())
        a, b = (np.abs(R.stochastic_e4m3(x, s, half, d)) for d in (-2.0 ** -16, 2.0 ** -16))
        if half is high:
            a, b = np.maximum(a, 2.0 ** -9), np.maximum(b, 2.0 ** -9)
        assert ((np.abs(got) >= a) & (np.abs(got) <= b)).all()


@GPU
@pytest.mark.parametrize("ct", ["f16", "bf16"])
def test_copies_beyond_half_the_last_cache(gpu, ct):
    """Above 128 MB of copies they are written past the caches: the same bits as of parts."""
    n, cut = 67_200_003, 33_600_001
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    p0, grad = torch.randn(n, generator=g, device="cuda") * 0.02, torch.randn(n, generator=g, device="cuda") * 1e-3
    got = []
    for parts in ([slice(0, n)], [slice(0, cut), slice(cut, n)]):
        p, c = p0.clone(), torch.empty(n, dtype=DT[ct], device="cuda")
        m, v = [], []
        for part in parts:
            opt = qcp.AdamW([p[part]], copies=[c[part]], state="f32")
            for step in (1, 2):
                qcp.adamw_step(opt, [grad[part]], step, **HYPER)
            k = part.stop - part.start
            m.append(opt.m[:k])
            v.append(opt.v[:k])
        got.append((p, c, torch.cat(m), torch.cat(v)))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and torch.equal(got[0][1], got[0][0].to(DT[ct]))


# bit patterns of NaN (quiet, all ones, negative) and of the infinities
BAD = {"f32": (0x7fc00000, 0x7fffffff, 0xffffffff, 0x7f800000, 0xff800000), "f16": (0x7e00, 0x7fff, 0xffff, 0x7c00, 0xfc00),
       "bf16": (0x7fc0, 0x7fff, 0xffff, 0x7f80, 0xff80)}


@GPU
@pytest.mark.parametrize("G", [0, 32, 128, 1024])
@pytest.mark.parametrize("gt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,where", [(5000, 2500), (777, 776)])
def test_a_gradient_that_is_not_finite_stays_visible(gpu, gt, G, n, where):
    """It makes its parameter NaN and, with 8-bit moments, the scales of its block,
    for good; every other block goes on as without it.  G = 0: fp32 moments."""
    one = G or 32
    block = slice(where // one * one, min((where // one + 1) * one, n)) if G else slice(where, where + 1)
    for pattern in BAD[gt]:
        seen = []
        for bad in (False, True):
            params, _ = flat_views([n], torch.float32, 1, 3, 0.02)
            opt = qcp.AdamW(params, state="e4m3" if G else "f32", G=one)
            for step in (1, 2, 3):
                g = flat_views([n], DT[gt], 1, 20 + step, 1e-2)[0][0]
                if bad and step == 2:
                    bits = g.view(torch.int32 if gt == "f32" else torch.int16)
                    bits[where] = pattern - (1 << (32 if gt == "f32" else 16)) if pattern >> (31 if gt == "f32" else 15) else pattern
                qcp.adamw_step(opt, [g], step, seed=7, **HYPER)
            seen.append((params[0].cpu(), opt.m.cpu(), opt.v.cpu(), *(s.cpu() for s in (opt.m_scales, opt.v_scales) if G)))
        (p0, *s0), (p1, *s1) = seen
        rest = torch.ones(n, dtype=torch.bool)
        rest[block] = False
        assert p1[block].isnan().all() and torch.equal(p1[rest], p0[rest]), (pattern, where)
        if G:
            mine = torch.zeros(len(s1[2]), dtype=torch.bool)
            mine[where // G] = True
            for a, b in zip(s0[2:], s1[2:]):
                assert b[mine].isnan().all() and torch.equal(a[~mine], b[~mine]), pattern
        for a, b in zip(s0[:2], s1[:2]):
            assert torch.equal(a[:n][rest], b[:n][rest]) and not b[n:].any(), pattern


@GPU
def test_a_variance_that_overflows_stays_visible(gpu):
    """A finite gradient whose square is beyond fp32: m stays finite, v does not."""
    n, G, where = 512, 64, 200
    params, _ = flat_views([n], torch.float32, 0, 3, 0.02)
    opt = qcp.AdamW(params, G=G)
    g = torch.full((n,), 1e-2, device="cuda")
    g[where] = 1e22
    qcp.adamw_step(opt, [g], 1, **HYPER)
    assert opt.v_scales.isnan().nonzero().flatten().tolist() == [where // G] and opt.m_scales.isfinite().all()
    assert params[0].isfinite().all()
    qcp.adamw_step(opt, [torch.full_like(g, 1e-2)], 2, **HYPER)
    assert params[0].isnan().nonzero().flatten().tolist() == list(range(192, 256))


@GPU
@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_the_smallest_eps(gpu, state):
    """eps = 2^-126, the least normal one, on zero gradients: nothing moves, nothing is NaN."""
    params, _ = flat_views([1000], torch.float32, 0, 3, 0.02)
    before = params[0].clone()
    opt = qcp.AdamW(params, state=state)
    for step in (1, 2):
        qcp.adamw_step(opt, [torch.zeros(1000, device="cuda")], step, lr=1e-3, eps=2.0 ** -126, weight_decay=0.0)
    assert torch.equal(params[0], before) and not opt.m.any() and not opt.v.any()


# ------------------------------------------------------------------ refusals (CPU)

OK, EINVAL, EALIGN = 0, -1, -2
A = 0x7f0000000000       # never dereferenced on these paths


def call(**kw):
    a = dict(params=[A], grads=[A + (1 << 30)], copies=None, sizes=[1024], offsets=[0], n=None, gt=3, ct=0,
             state=0x43, m=A + (2 << 30), ms=A + (3 << 30), v=A + (4 << 30), vs=A + (5 << 30), n_state=1024,
             G=128, step=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, scale=None, seed=0)
    a.update(kw)
    k = len(a["sizes"])
    ptrs = lambda x: None if x is None else (ctypes.c_void_p * k)(*x)  # noqa: E731
    return qcp.library().adamw_step(
        ptrs(a["params"]), ptrs(a["grads"]), ptrs(a["copies"]), (ctypes.c_int64 * k)(*a["sizes"]),
        (ctypes.c_int64 * k)(*a["offsets"]), k if a["n"] is None else a["n"], a["gt"], a["ct"], a["state"],
        a["m"], a["ms"], a["v"], a["vs"], a["n_state"], a["G"], a["step"], a["lr"], a["b1"], a["b2"], a["eps"],
        a["wd"], a["scale"], a["seed"], None)


@pytest.fixture()
def lib():
    if not os.path.exists(qcp.LIB_PATH):
        pytest.fail(f"{qcp.LIB_PATH} not built")


def test_c_entry_refuses(lib):
    assert call(n=0) == OK and call(sizes=[0]) == OK                  # nothing to do, no launch
    for bad in (dict(n=-1), dict(n=1025), dict(G=100), dict(gt=0), dict(gt=9), dict(state=8), dict(step=0),
                dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(b1=1.0), dict(b1=-0.1),
                dict(b2=1.0), dict(b2=float("nan")), dict(eps=0.0), dict(eps=1e-60), dict(eps=float("nan")),
                dict(wd=-0.1), dict(wd=float("inf")), dict(sizes=[-1]), dict(sizes=[1 << 40]),
                dict(n_state=1023), dict(n_state=-1), dict(sizes=[1025]), dict(offsets=[-128]),
                dict(offsets=[64]), dict(offsets=[1 << 62]), dict(params=[0]), dict(grads=[0]), dict(m=0),
                dict(v=None), dict(ms=0), dict(vs=0), dict(copies=[A + (6 << 30)], ct=3),
                dict(copies=[0], ct=2)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(params=[A + 2]), dict(grads=[A + (1 << 30) + 2]), dict(grads=[A + (1 << 30) + 1], gt=1),
                dict(m=A + (2 << 30) + 4), dict(vs=A + (5 << 30) + 8), dict(copies=[A + (6 << 30) + 1], ct=2),
                dict(scale=A + (7 << 30) + 2)):
        assert call(**bad) == EALIGN, bad
    # overlaps: a written buffer with any other, moments and factors among them
    for bad in (dict(grads=[A + 64]), dict(m=A), dict(v=A + (2 << 30) + 512), dict(ms=A + (5 << 30)),
                dict(copies=[A + 2048], ct=2), dict(scale=A + 128), dict(vs=A + (1 << 30))):
        assert call(**bad) == EINVAL, bad
    two = dict(sizes=[1024, 1024], n_state=2048, grads=[A + (1 << 30)] * 2)
    assert call(**two, params=[A, A + 4092], offsets=[0, 1024]) == EINVAL
    assert call(**two, params=[A + 4000, A], offsets=[0, 1024]) == EINVAL     # in either order
    assert call(**two, params=[A, A + 4096], offsets=[1024, 0]) == EINVAL     # offsets descend
    assert call(**two, params=[A, A + 4096], offsets=[0, 896]) == EINVAL      # blocks overlap


def test_binding_refuses(lib):
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt)  # noqa: E731

    def raises(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)
    raises("list of tensors", qcp.AdamW, f(8))
    raises("empty list", qcp.AdamW, [])
    raises("params\\[1\\]: dtype", qcp.AdamW, [f(8), f(8, torch.bfloat16)])
    raises("params\\[0\\]: must be contiguous", qcp.AdamW, [f(16)[::2]])
    raises("state 'int8'", qcp.AdamW, [f(8)], state="int8")
    raises("block size", qcp.AdamW, [f(8)], G=48)
    raises("copies: 1 tensors for 2", qcp.AdamW, [f(8), f(8)], copies=[f(8, torch.float16)])
    raises("copies\\[0\\]: dtype", qcp.AdamW, [f(8)], copies=[f(8)])
    raises("copies\\[1\\]: dtype", qcp.AdamW, [f(8), f(8)], copies=[f(8, torch.float16), f(8, torch.bfloat16)])
    raises("copies\\[0\\]: holds 7", qcp.AdamW, [f(8)], copies=[f(7, torch.float16)])
    raises("m: holds", qcp.AdamW, [f(200)], m=f(255, torch.uint8))
    raises("m: dtype", qcp.AdamW, [f(200)], m=f(256))
    raises("v_scales: holds", qcp.AdamW, [f(200)], v_scales=f(1))
    raises("GPU tensors only", qcp.AdamW, [f(8)])


@GPU
def test_step_refuses(gpu):
    z = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    p = z(300)
    opt = qcp.AdamW([p, z(5)], state="f32")

    def raises(match, grads, **kw):
        with pytest.raises(ValueError, match=match):
            qcp.adamw_step(opt, grads, 1, 1e-3, **kw)
    raises("1 tensors for 2", [z(300)])
    raises("list of tensors", z(300))
    raises("grads\\[0\\]: dtype", [z(300, torch.float64), z(5)])
    raises("grads\\[1\\]: dtype", [z(300), z(5, torch.float16)])
    raises("grads\\[1\\]: holds 4", [z(300), z(4)])
    raises("grads\\[1\\]: holds 6", [z(300), z(6)])
    raises("must be contiguous", [z(600)[::2], z(5)])
    raises("expected a torch.Tensor", [z(300), None])
    raises("GPU tensors only", [z(300), torch.zeros(5)])
    raises("grad_scale: dtype", [z(300), z(5)], grad_scale=z(1, torch.float64))
    with pytest.raises(qcp.QcpError):
        qcp.adamw_step(opt, [z(300), z(5)], 0, 1e-3)
    p.data = z(300)
    raises("another storage", [z(300), z(5)])


def test_c_entry_refuses_an_eps_below_normal(lib):
    """1/(0 + eps) has to be finite in fp32, and the device's reciprocal takes what is
    below 2^-126 for 0."""
    for eps in (1e-45, 1e-40, 2.0 ** -127, np.nextafter(2.0 ** -126, 0)):
        want = EINVAL if np.float32(eps) < np.float32(2.0 ** -126) else OK
        assert call(eps=float(eps), sizes=[0]) == want, eps


# ------------------------------------------------------------------ tensors that moved


@pytest.fixture()
def on_cpu(monkeypatch):
    """The binding on CPU tensors, with the launch replaced: the list of calls it would make."""
    from quantized_collective_payloads_amd import optimizer
    calls = []
    monkeypatch.setattr(optimizer, "_dev", lambda *ts: torch.device("cpu"))
    monkeypatch.setattr(optimizer, "_enqueue", lambda name, index, *args: calls.append((name, args)))
    return calls


def small(device, state="e4m3", separate=True):
    """An AdamW over two tensors with everything that a step reads or writes given to it."""
    z = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device=device)  # noqa: E731
    eight = state == "e4m3"
    kind = torch.uint8 if eight else torch.float32
    params = [z(300), z(5)] if separate else list(z(305).split([300, 5]))
    opt = qcp.AdamW(params, copies=[z(300, torch.bfloat16), z(5, torch.bfloat16)], state=state, m=z(512, kind),
                    v=z(512, kind), m_scales=z(4) if eight else None, v_scales=z(4) if eight else None)
    return opt, [z(300), z(5)]


def tensors_of(opt):
    got = {f"params[{i}]": p for i, p in enumerate(opt.params)} | {f"copies[{i}]": c for i, c in enumerate(opt.copies)}
    got |= {"m": opt.m, "v": opt.v}
    return got | ({} if opt.m_scales is None else {"m_scales": opt.m_scales, "v_scales": opt.v_scales})


# how a tensor comes to lie elsewhere, or to hold less than it did where it was
MOVES = {"data": lambda t: setattr(t, "data", t.clone()), "set": lambda t: t.set_(t.clone()),
         "freed": lambda t: t.untyped_storage().resize_(0),
         "shrunk": lambda t: t.untyped_storage().resize_(t.untyped_storage().nbytes() // 2)}


@pytest.mark.parametrize("how", MOVES)
@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_a_tensor_with_another_storage_is_refused(on_cpu, state, how):
    names = list(tensors_of(small("cpu", state)[0]))
    assert len(names) == (8 if state == "e4m3" else 6)
    for name in names:
        opt, grads = small("cpu", state)
        qcp.adamw_step(opt, grads, 1, 1e-3)
        assert len(on_cpu) == 1
        on_cpu.clear()
        MOVES[how](tensors_of(opt)[name])
        with pytest.raises(ValueError, match=f"^{name.replace('[', '.').replace(']', '.')}: given another storage"):
            qcp.adamw_step(opt, grads, 2, 1e-3)
        assert not on_cpu


def test_a_storage_shared_by_several_tensors_is_named_for_each(on_cpu):
    opt, grads = small("cpu", separate=False)
    qcp.adamw_step(opt, grads, 1, 1e-3)
    opt.params[0].untyped_storage().resize_(1240)                  # more than it was
    with pytest.raises(ValueError, match="params.0., params.1.: given another storage"):
        qcp.adamw_step(opt, grads, 2, 1e-3)
    assert len(on_cpu) == 1


@GPU
def test_a_moved_copy_is_not_written(gpu):
    """What the copies and moments were given instead, and where they were, stays as it is."""
    for name in ("copies[0]", "m", "v_scales"):
        opt, grads = small("cuda")
        t = tensors_of(opt)[name]
        old, new = t.detach(), torch.ones_like(t)
        t.data = new
        with pytest.raises(ValueError, match="another storage"):
            qcp.adamw_step(opt, [g + 1 for g in grads], 1, 1e-3)
        torch.cuda.synchronize()
        assert not old.any() and (new == 1).all() and not opt.params[0].any(), name


@pytest.mark.parametrize("state", ["e4m3", "f32"])
def test_every_written_tensor_gets_a_new_version(on_cpu, state):
    opt, grads = small("cpu", state)
    before = {name: t._version for name, t in tensors_of(opt).items()}
    qcp.adamw_step(opt, grads, 1, 1e-3)
    assert all(t._version > before[name] for name, t in tensors_of(opt).items())


def test_a_step_after_a_moment_entered_a_graph_is_seen(on_cpu):
    opt, grads = small("cpu", "f32")
    w = torch.ones(512, requires_grad=True)
    y = (w * opt.m).sum()
    qcp.adamw_step(opt, grads, 1, 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


# ------------------------------------------------------------------ more tensors than one call takes


def check(n, **kw):
    """qcp_adamw_check for n tensors of 4 elements (G = 32) at addresses of their own."""
    base = {"params": A, "grads": A + (1 << 30), "copies": A + (2 << 30)}
    a = {k: [b + 64 * i for i in range(n)] for k, b in base.items()}
    a |= dict(sizes=[4] * n, offsets=[32 * i for i in range(n)], gt=3, ct=2, state=0x43, m=A + (3 << 30), ms=A + (4 << 30),
              v=A + (5 << 30), vs=A + (6 << 30), n_state=32 * n, G=32, step=1, eps=1e-8, scale=A + (7 << 30))
    for k, v in kw.items():
        if isinstance(v, dict):                                    # one place of an array
            for i, x in v.items():
                a[k][i] = x
        else:
            a[k] = v
    arr = lambda t, x: None if x is None else (t * n)(*x)  # noqa: E731
    return qcp.library().qcp_adamw_check(
        *(arr(ctypes.c_void_p, a[k]) for k in ("params", "grads", "copies")), arr(ctypes.c_int64, a["sizes"]),
        arr(ctypes.c_int64, a["offsets"]), n, a["gt"], a["ct"], a["state"], a["m"], a["ms"], a["v"], a["vs"],
        a["n_state"], a["G"], a["step"], 1e-3, 0.9, 0.999, a["eps"], 0.0, a["scale"])


@pytest.mark.parametrize("n", [6, 1024, 2100])
def test_check_over_any_number_of_tensors(lib, n):
    first, last = 1, n - 2
    assert check(n) == OK and check(n, copies=None) == OK and check(n, scale=None) == OK
    assert check(n, sizes=[0] * n, params=[0] * n) == OK           # nothing to do
    # gradients may meet one another
    assert check(n, grads={first: A + (1 << 30) + 64 * last}) == OK
    for bad in (dict(params={first: A + 64 * last + 12}), dict(params={last: A + 64 * first}),
                dict(grads={last: A + 64 * first + 8}), dict(grads={first: A + (3 << 30) + 32 * last}),
                dict(copies={last: A + 64 * first}), dict(copies={first: A + (2 << 30) + 64 * last + 2}),
                dict(scale=A + 64 * last), dict(m=A), dict(v=A + (3 << 30)), dict(params={last: 0}), dict(copies={last: 0}),
                dict(sizes={last: -1}), dict(sizes={last: 33}), dict(offsets={last: 0}), dict(n_state=32 * n - 1),
                dict(step=0), dict(eps=0.0), dict(G=33), dict(gt=9), dict(state=1), dict(ct=3)):
        assert check(n, **bad) == EINVAL, bad
    for bad in (dict(params={last: A + 64 * last + 2}), dict(copies={last: A + (2 << 30) + 64 * last + 1}),
                dict(vs=A + (6 << 30) + 8), dict(scale=A + (7 << 30) + 1)):
        assert check(n, **bad) == EALIGN, bad


def test_check_without_arguments(lib):
    c = qcp.library().qcp_adamw_check
    none = [None] * 5
    rest = (3, 2, 0x43, None, None, None, None, 0, 32, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0, None)
    assert c(*none, 0, *rest) == OK and c(*none, -1, *rest) == EINVAL and c(*none, 1 << 62, *rest) == EINVAL


def many(device, n=2100):
    z = lambda k: torch.zeros(k, device=device)  # noqa: E731
    opt = qcp.AdamW([z(8) for _ in range(n)], state="f32", G=32)
    return opt, [z(8) + 1 for _ in range(n)]


BROKEN = {"a parameter twice, far apart": lambda p, g: p.__setitem__(1500, p[5]),
          "a later gradient that is an earlier parameter": lambda p, g: g.__setitem__(2000, p[3]),
          "an earlier gradient that is a later parameter": lambda p, g: g.__setitem__(3, p[2000]),
          "a gradient that is its parameter, in the last call": lambda p, g: g.__setitem__(2060, p[2060])}


@pytest.mark.parametrize("what", BROKEN)
def test_a_step_of_several_calls_is_refused_whole(on_cpu, lib, what):
    opt, grads = many("cpu")
    params = list(opt.params)
    BROKEN[what](params, grads)
    opt = qcp.AdamW(params, state="f32", G=32)
    with pytest.raises(qcp.QcpError, match="adamw_step"):
        qcp.adamw_step(opt, grads, 1, 1e-3)
    assert not on_cpu and params[7]._version == 0
    opt, grads = many("cpu")
    qcp.adamw_step(opt, grads, 1, 1e-3)
    assert [args[5] for _, args in on_cpu] == [1024, 1024, 52]


@GPU
@pytest.mark.parametrize("what", BROKEN)
def test_a_refused_step_of_several_calls_changes_nothing(gpu, what):
    opt, grads = many("cuda")
    params = list(opt.params)
    BROKEN[what](params, grads)
    opt = qcp.AdamW(params, state="f32", G=32)
    with pytest.raises(qcp.QcpError, match="adamw_step"):
        qcp.adamw_step(opt, grads, 1, 1e-3)
    torch.cuda.synchronize()
    assert not opt.m.any() and not opt.v.any() and not torch.cat(params).any()
