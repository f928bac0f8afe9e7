"""Sizes and uses of the layer operators that reach their further code paths:
large counts, other streams, graphs of bound calls, kernels chosen for many
tokens.  Bounds and helpers are those of test_gpu_layer."""
import ctypes

import numpy as np
import pytest
import torch

import workloads
from oracle import layer as ref
from test_gpu_layer import HALF, TINY, U, Gated, check_gated, f64, near, normal, shifted

csf = pytest.importorskip("moe_weight_decode_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("S", [3_000_000, 4_194_304 + 37])
def test_millions_of_slots_of_one_expert(dev, S):
    # blocks of 16 slots times tiles passes 32 bits; every slot's result is its token's
    F, K, T = 16, 32, 1000
    c = Gated(1, F, K, [T], workloads.NVFP4, seed=21, T=T)
    token = torch.arange(T, dtype=torch.int32, device=dev)
    h, gu = csf.moe_gated(c.stack, c.tw, c.x, c.ta, c.te, token, save=True)
    dh = normal(np.random.default_rng(3), T, F, dtype=torch.bfloat16)
    dx, dgu = csf.moe_gated_backward(c.stack, c.dense(), c.tw, dh, gu, c.ta, c.te)
    rows = token.repeat((S + T - 1) // T)[:S].contiguous()
    es, at = torch.tensor([0, S], dtype=torch.int32, device=dev), rows.long()
    hs, gus = csf.moe_gated(c.stack, c.tw, c.x, c.ta, es, rows, save=True)
    assert torch.equal(hs, h[at]) and torch.equal(gus, gu[at])
    dxs, dgus = csf.moe_gated_backward(c.stack, c.dense(), c.tw, dh[at], gus, c.ta, es)
    assert torch.equal(dxs, dx[at]) and torch.equal(dgus, dgu[at])


def test_gated_backward_of_millions_of_rows(dev):
    # 128 slots of 2F = 9,000,032 rows: 2.3 GB of dgu in a tile, past 31-bit offsets.  The last step of 64 rows is half
    # full; what its other half reads must be 0 for every slot, whatever stands in another slot's rows.
    S, N, K = 128, 9_000_032, 32
    F = N // 2
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    gu = torch.randn(S, N, generator=g, device=dev, dtype=torch.bfloat16)
    dh = torch.randn(S, F, generator=g, device=dev, dtype=torch.bfloat16)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    dense = torch.full((N,), 127, dtype=torch.uint8, device=dev)
    es, alpha = torch.tensor([0, S], dtype=torch.int32, device=dev), torch.full((1,), 0.25, device=dev)
    d = csf.csf_stack()
    d.format, d.num_experts, d.rows, d.cols = csf.MXFP4, 1, N, 1

    def backward():
        dx, dgu = torch.empty(S, K, dtype=torch.bfloat16, device=dev), torch.empty(S, N, dtype=torch.bfloat16, device=dev)
        assert csf.library().csf_moe_gated_backward(
            ctypes.byref(d), dense.data_ptr(), codes.data_ptr(), dh.data_ptr(), gu.data_ptr(), S, alpha.data_ptr(), es.data_ptr(),
            dx.data_ptr(), dgu.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        return dx, dgu

    dx, dgu = backward()
    table = torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0), device=dev)
    w = table[torch.stack((codes & 15, codes >> 4), 2).flatten(1).int()].double()
    for s in (0, 127):
        v = dgu[s].double()
        want, mag = 0.25 * (v @ w), 0.25 * (v.abs() @ w.abs())
        # a running sum is rounded once per 32 rows, and a product's 32 terms add their own roundings
        near(dx[s], f64(want), 2.0 ** -8 * np.abs(f64(want)) + (N // 32 + 40) * U * f64(mag), "dx")
    del w, dgu
    gu[120] = float("nan")
    bad, _ = backward()
    assert bad[120].isnan().all() and torch.equal(bad[:120], dx[:120]) and torch.equal(bad[121:], dx[121:])


def test_gated_backward_writes_routed_slots_only(dev):
    # routing of some of the experts, as of one device's: the slots before the first one's are others'
    c = Gated(3, 40, 96, [4, 3, 9], workloads.NVFP4, seed=4)
    S, first = len(c.rows), 4
    _, gu = c.forward(save=True)
    dh = normal(np.random.default_rng(5), S, c.F, dtype=torch.bfloat16)
    want = csf.moe_gated_backward(c.stack, c.dense(), c.tw, dh, gu, c.ta, c.te)
    es = c.te.clone()
    es[0] = first  # expert 0 has no slots left
    gu[:first] = float("nan")
    d = c.stack.descriptor()
    dx = torch.full((S, c.K), 7.0, dtype=torch.bfloat16, device=dev)
    dgu = torch.full((S, 2 * c.F), 7.0, dtype=torch.bfloat16, device=dev)
    assert csf.library().csf_moe_gated_backward(
        ctypes.byref(d), c.dense().data_ptr(), c.tw.data_ptr(), dh.data_ptr(), gu.data_ptr(), S, c.ta.data_ptr(), es.data_ptr(),
        dx.data_ptr(), dgu.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    for got, full in ((dx, want[0]), (dgu, want[1])):
        assert (got[:first] == 7).all() and torch.equal(got[first:], full[first:])


KINDS = {"nvfp4": (workloads.NVFP4, False), "mxfp4": (workloads.MXFP4, False), "mx8": (workloads.MXFP4, True)}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("E,F,K,counts", [
    (3, 24, 5120, [1, 0, 17]), (2, 20, 8192, [2, 19]), (2, 17, 4128, [1, 1]),  # more than 4 chunks of K a wave
    (40, 24, 64, [15] * 40),                                                   # more slots than come with the routing
    (300, 9, 96, [0, 1, 2] * 100),
    (9, 33, 1056, [0, 40, 0, 1, 0, 90, 3, 0, 16]),                             # few slots over all, many of one expert
])
def test_gated_few_slots(dev, E, F, K, counts, kind):
    assert sum(counts) < 20 * E
    fmt, x8 = KINDS[kind]
    c = Gated(E, F, K, counts, fmt, x8, seed=E + F + K)
    h, gu = c.forward(save=True)
    check_gated(c, h, gu)
    assert torch.equal(c.forward(), h)
    h2, gu2 = c.forward(save=True, dense_scales=c.dense())
    assert torch.equal(h2, h) and torch.equal(gu2, gu)


@pytest.mark.parametrize("kind", KINDS)
def test_few_slots_with_nan_tokens(dev, kind):
    fmt, x8 = KINDS[kind]
    c = Gated(3, 40, 160, [5, 0, 30], fmt, x8, seed=9, T=12)
    clean = c.forward()
    c.x[3] = 0x7f if x8 else float("nan")
    h = c.forward()
    hit = torch.from_numpy(c.rows == 3).to(dev)
    assert hit.any() and h[hit].isnan().all() and torch.equal(h[~hit], clean[~hit])


@pytest.mark.parametrize("kind", KINDS)
def test_tiles_without_their_counters(dev, kind):
    # scales decoded beforehand and no workspace: the tiles are dealt out in turn
    fmt, x8 = KINDS[kind]
    c = Gated(5, 300, 96, [1, 0, 700, 16, 300], fmt, x8, seed=31)
    h, gu = c.forward(save=True)
    check_gated(c, h, gu)
    d, dense, S = c.stack.descriptor(), c.dense(), len(c.rows)
    out, ogu = torch.empty_like(h), torch.empty_like(gu)
    assert csf.library().csf_moe_gated(
        ctypes.byref(d), dense.data_ptr(), c.tw.data_ptr(), c.x.data_ptr(), c.xs.data_ptr() if x8 else None, c.x.shape[0],
        c.ta.data_ptr(), c.te.data_ptr(), c.tr.data_ptr(), S, out.data_ptr(), ogu.data_ptr(), None, 0,
        torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, h) and torch.equal(ogu, gu)


@pytest.mark.parametrize("counts", [[3, 0, 8], [70, 0, 130]])
@pytest.mark.parametrize("F", [40, 41])
def test_gated_tensors_at_their_least_alignment(dev, F, counts):
    c = Gated(3, F, 96, counts, workloads.NVFP4, seed=35)
    S, lib, stream = len(c.rows), csf.library(), torch.cuda.current_stream().cuda_stream
    h, gu = c.forward(save=True)
    dh = normal(np.random.default_rng(2), S, F, dtype=torch.bfloat16)
    dx, dgu = csf.moe_gated_backward(c.stack, c.dense(), c.tw, dh, gu, c.ta, c.te)
    d, alpha, es, rows = c.stack.descriptor(), shifted(c.ta, 1), shifted(c.te, 1), shifted(c.tr, 1)
    need = lib.csf_moe_gated_workspace(ctypes.byref(d), S)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    out, ogu, odgu = shifted(torch.zeros_like(h), 1), shifted(torch.zeros_like(gu), 1), shifted(torch.zeros_like(dgu), 2)
    odx, dense = torch.zeros_like(dx), shifted(c.dense(), 1)
    assert lib.csf_moe_gated(ctypes.byref(d), None, c.tw.data_ptr(), c.x.data_ptr(), None, c.x.shape[0], alpha.data_ptr(),
                             es.data_ptr(), rows.data_ptr(), S, out.data_ptr(), ogu.data_ptr(), ws.data_ptr(), need, stream) == 0
    assert torch.equal(out, h) and torch.equal(ogu, gu)
    assert lib.csf_moe_gated(ctypes.byref(d), dense.data_ptr(), c.tw.data_ptr(), c.x.data_ptr(), None, c.x.shape[0],
                             alpha.data_ptr(), es.data_ptr(), rows.data_ptr(), S, out.data_ptr(), ogu.data_ptr(), None, 0, stream) == 0
    assert torch.equal(out, h) and torch.equal(ogu, gu)
    dh, gu = shifted(dh, 1), shifted(gu, 1)
    assert lib.csf_moe_gated_backward(ctypes.byref(d), dense.data_ptr(), c.tw.data_ptr(), dh.data_ptr(), gu.data_ptr(), S,
                                      alpha.data_ptr(), es.data_ptr(), odx.data_ptr(), odgu.data_ptr(), stream) == 0
    assert torch.equal(odx, dx) and torch.equal(odgu, dgu)


@pytest.mark.parametrize("kind", KINDS)
def test_activations_past_31_bit_offsets(dev, kind):
    # more activations than a tile's offsets reach: many slots, taken as few are
    fmt, x8 = KINDS[kind]
    c = Gated(2, 40, 32, [70, 90], fmt, x8, seed=33, T=100)
    T = (2 ** 31 // 32 if x8 else 2 ** 31 // 64) + 1000
    rng = np.random.default_rng(5)
    at = torch.from_numpy(np.sort(rng.choice(T - 1, 99, replace=False)).astype(np.int32)).to(dev)
    at = torch.cat((at, torch.tensor([T - 1], dtype=torch.int32, device=dev)))
    x = torch.zeros(T, 32, dtype=c.x.dtype, device=dev)
    x[at.long()] = c.x
    if x8:
        xs = torch.zeros(T, 1, dtype=torch.uint8, device=dev)
        xs[at.long()] = c.xs
        c.xs = xs
    c.x, c.tr = x, at[c.tr.long()]
    h, gu = c.forward(save=True)
    check_gated(c, h, gu)


# ------------------------------------------------------------------ many tokens

def route_of_many(logits, k, renorm):
    """oracle.layer.route for many tokens at once."""
    l = np.where(np.isnan(logits), -np.inf, logits)
    T, E = l.shape
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(l, order, 1)
    on = top > -np.inf
    experts = np.where(on, order, -1)
    most = np.where(on[:, :1], top[:, :1], 0.0)
    p = np.where(on, np.exp(top - most), 0.0)
    whole = p.sum(1, keepdims=True) if renorm else np.exp(l - most).sum(1, keepdims=True)
    gates = np.where(on, p / np.where(on[:, :1], whole, 1.0), 0.0)
    flat = np.where(experts < 0, E, experts).reshape(-1)
    by = np.argsort(flat, kind="stable")
    start = np.searchsorted(flat[by], np.arange(E + 1))
    rows, slots = np.full(T * k, -1), np.full(T * k, -1)
    rows[:start[E]] = by[:start[E]] // k
    slots[by[:start[E]]] = np.arange(start[E])
    return experts, gates, start, rows, slots.reshape(T, k)


def same_routing(r, want, k, E, renorm):
    e, g, start, rows, slots = want
    assert np.array_equal(r.experts.cpu().numpy(), e) and np.array_equal(r.expert_start.cpu().numpy(), start)
    assert np.array_equal(r.rows.cpu().numpy(), rows) and np.array_equal(r.slots.cpu().numpy(), slots)
    near(r.gates, g, ((k if renorm else E) + 24) * U * g, "gates")


def test_the_oracle_of_many_is_the_oracle(dev):
    rng = np.random.default_rng(1)
    l = rng.integers(-3, 3, (90, 11)).astype(np.float64)  # many equal ones
    l[rng.random(l.shape) < 0.3] = -np.inf
    l[7], l[8, 3] = -np.inf, np.nan
    for renorm in (True, False):
        for a, b in zip(route_of_many(l, 4, renorm), ref.route(l, 4, renorm)):
            assert np.allclose(a, b, rtol=1e-14, atol=0)


# 16 lanes a token from 2048 tokens on (2, 4, 8, 16, 24 or 32 logits a lane), 64 above 512 experts or 16 choices;
# workgroups' counts added up by each up to 16384 tokens, by a kernel of their own beyond
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(2048, 33, 3), (2049, 2, 2), (2049, 65, 16), (2047, 100, 4), (2111, 256, 8), (4100, 384, 8),
                                   (2100, 512, 16), (2050, 513, 3), (2060, 64, 17), (2048, 16, 1), (16384, 40, 2),
                                   (16385, 40, 2), (20000, 7, 3), (17000, 600, 2)])
def test_route_of_many_tokens(dev, T, E, k, dtype):
    rng = np.random.default_rng(T + 31 * E + k)
    logits = normal(rng, T, E, dtype=dtype, scale=1.5)
    masked = logits.masked_fill(torch.from_numpy(rng.random((T, E)) < 0.3).to(dev), float("-inf"))
    masked[T // 2] = float("-inf")
    masked[T - 1, 1:] = float("nan")
    for renorm in (True, False):
        for l in (logits, masked):
            want = route_of_many(f64(l.float()), k, renorm)
            same_routing(csf.route(l, k, renorm=renorm), want, k, E, renorm)
    equal = torch.zeros(T, E, dtype=dtype, device=dev)
    equal[:, ::2] = -0.0
    assert torch.equal(csf.route(equal, k).experts, torch.arange(k, dtype=torch.int32, device=dev).expand(T, k))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_masked_logits_get_no_gradient_whatever_the_gates_get(dev, value, renorm):
    rng = np.random.default_rng(41)
    T, E, k = 9, 130, 4
    logits = normal(rng, T, E).masked_fill(torch.from_numpy(rng.random((T, E)) < 0.4).to(dev), float("-inf"))
    logits[7] = float("nan")
    r = csf.route(logits, k, renorm=renorm)
    dg = normal(rng, T, k)
    clean = csf.route_backward(dg, logits, r.experts, r.gates, renorm=renorm)
    dg[3, 1] = value
    dg[7] = value  # of no choice
    got = csf.route_backward(dg, logits, r.experts, r.gates, renorm=renorm)
    masked = ~(logits > float("-inf"))
    assert (got[masked] == 0).all()
    others = torch.arange(T, device=dev) != 3
    assert torch.equal(got[others], clean[others]) and not got[3].isfinite().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(9000, 24), (4100, 1000), (3100, 1030), (1100, 8200), (1030, 20000)])
def test_norm_backward_of_many_tokens(dev, T, D, dtype):
    # several rows to a workgroup, its two buffers of partial sums in turn
    rng = np.random.default_rng(T + D)
    total, dy, ds = (normal(rng, T, D, dtype=dtype) for _ in range(3))
    w = 1.0 + normal(rng, D, scale=0.1)
    rstd = csf.rms_norm(total, w).rstd
    dx, dw = csf.rms_norm_backward(dy, total, w, rstd, dsum=ds)
    wx, ww, mx, mw = ref.rms_norm_backward(f64(dy), f64(total), f64(w), f64(rstd), f64(ds))
    near(dx, wx, HALF[dtype] * np.abs(wx) + (D + 16) * U * mx * (1 + HALF[dtype]) + TINY[dtype], "dx")
    near(dw, ww, (T + 16) * U * mw, "dweight")


# ------------------------------------------------------------------ launches past 2^32 threads

MANY = 2 ** 26 + 5  # tokens of a wave each


def ends(T):
    """Tokens at both ends and around the first that a launch of one axis would not reach."""
    return [slice(0, 300), slice(2 ** 26 - 150, min(T, 2 ** 26 + 150)), slice(T - 300, T)]


def test_norm_of_more_tokens_than_a_launch_axis_holds(dev):
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    x = torch.randn(MANY, 4, generator=g, device=dev, dtype=torch.bfloat16)
    w = torch.tensor([0.5, 1.0, 2.0, 3.0], device=dev)
    r = csf.rms_norm(x, w)
    for s in ends(MANY):
        want = csf.rms_norm(x[s].contiguous(), w)
        assert torch.equal(r.out[s], want.out) and torch.equal(r.rstd[s], want.rstd)
    assert (r.rstd > 0).all()


def test_norm_of_more_long_rows_than_a_launch_axis_holds(dev):
    # a workgroup a row: 2^24 rows of 256 threads; the sums of few experts' outputs, as 8 bits, to keep it small
    T, D, S = 2 ** 24 + 3, 1025, 5
    rng = np.random.default_rng(7)
    x, w, gates = normal(rng, S, D), 1.0 + normal(rng, D, scale=0.1), torch.ones(T, 1, device=dev)
    slots = (torch.arange(T, dtype=torch.int32, device=dev) % S)[:, None].contiguous()
    out = torch.zeros(T, D, dtype=torch.uint8, device=dev)
    scales, rstd = torch.zeros(T, 33, dtype=torch.uint8, device=dev), torch.zeros(T, device=dev)
    assert csf.library().csf_rms_norm(0, x.data_ptr(), None, w.data_ptr(), T, D, slots.data_ptr(), gates.data_ptr(), 1, S, 1e-6,
                                      None, out.data_ptr(), scales.data_ptr(), rstd.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream) == 0
    want = csf.rms_norm(x, w, mxfp8=True)
    assert torch.equal(rstd, want.rstd[slots[:, 0].long()])
    for at in (0, 2 ** 24 - 5, T - 5):
        k = slots[at:at + 5, 0].long()
        assert torch.equal(out[at:at + 5], want.out[k]) and torch.equal(scales[at:at + 5], want.scales[k])


def test_route_and_gradients_of_more_tokens_than_a_launch_axis_holds(dev):
    g = torch.Generator(device=dev)
    g.manual_seed(8)
    logits = torch.randn(MANY, 2, generator=g, device=dev)
    y, dout = torch.randn(MANY, 2, generator=g, device=dev), torch.randn(MANY, 2, generator=g, device=dev, dtype=torch.bfloat16)
    slots = torch.arange(MANY, dtype=torch.int32, device=dev)[:, None].contiguous()
    gates = torch.rand(MANY, 1, generator=g, device=dev)
    dy, dg = csf.combine_backward(dout, y, slots, gates)
    experts = (logits[:, :1] < logits[:, 1:]).to(torch.int32)
    dl = csf.route_backward(dg, logits, experts, gates, renorm=False)
    for s in ends(MANY):
        n = s.stop - s.start
        want = csf.combine_backward(dout[s].contiguous(), y[s].contiguous(), slots[:n].contiguous(), gates[s].contiguous())
        assert torch.equal(dy[s], want[0]) and torch.equal(dg[s], want[1])
        want = csf.route_backward(dg[s].contiguous(), logits[s].contiguous(), experts[s].contiguous(), gates[s].contiguous(), renorm=False)
        assert torch.equal(dl[s], want)


def test_route_of_more_tokens_than_a_launch_axis_holds(dev):
    # 1024 threads for 64 tokens
    T = 2 ** 28 + 70
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    logits = torch.randn(T, 2, generator=g, device=dev, dtype=torch.bfloat16)
    r = csf.route(logits, 1)
    second = logits[:, 0] < logits[:, 1]
    assert torch.equal(r.experts[:, 0], second.to(torch.int32)) and (r.gates == 1).all()
    zeros = T - int(second.sum())
    assert r.expert_start.tolist() == [0, zeros, T]
    token = torch.arange(T, dtype=torch.int32, device=dev)
    order = torch.cat((token[~second], token[second]))
    assert torch.equal(r.rows, order)
    assert torch.equal(r.slots[order.long(), 0], token)


# ------------------------------------------------------------------ 8-bit activations

def any_codes(rng, c: Gated):
    """Every E4M3 code but NaN alike often, the scales 2^-5 .. 2^5: products of one
    sum that lie up to 2^22 apart, and their sums often near 0."""
    T = c.x.shape[0]
    codes = rng.integers(0, 256, (T, c.K)).astype(np.uint8)
    codes[codes & 0x7f == 0x7f] = 0
    scales = rng.integers(122, 133, (T, c.K // 32)).astype(np.uint8)
    c.x, c.xs = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    c.x64 = f64(c.x.view(torch.float8_e4m3fn).float()) * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=1)
    return c


@pytest.mark.parametrize("E,F,K,counts", [
    (2, 40, 32, [3, 16]), (2, 200, 32, [130, 90]),              # few slots, many
    (3, 33, 160, [7, 0, 18]), (2, 129, 160, [257, 20]),
    (8, 16, 2048, [1, 2, 0, 3, 1, 1, 17, 5]), (1, 64, 2048, [64]),
    (2, 24, 5120, [4, 19]), (1, 20, 8192, [31]),
])
def test_sums_of_any_8_bit_codes_are_as_in_float32(dev, E, F, K, counts):
    rng = np.random.default_rng(E + F + K)
    c = any_codes(rng, Gated(E, F, K, counts, workloads.MXFP4, True, seed=F + K))
    h, gu = c.forward(save=True)
    check_gated(c, h, gu)


def test_many_experts_by_tiles_with_8_bit_activations(dev):
    rng = np.random.default_rng(8)
    counts = rng.integers(0, 45, 700)
    counts[[0, 3, 4, 5, 699]] = 0
    counts[350] = 300
    c = Gated(700, 9, 32, counts, workloads.MXFP4, True, seed=16)
    for codes in (c, any_codes(rng, c)):
        h, gu = codes.forward(save=True)
        check_gated(codes, h, gu)
        assert torch.equal(codes.forward(dense_scales=codes.dense()), h)


# ------------------------------------------------------------------ streams and graphs

def test_inputs_dropped_after_a_call_on_another_stream(dev):
    """Inputs freed when the call returns, `stream` still busy: what the current
    stream allocates and writes next must not be their memory."""
    rng = np.random.default_rng(17)
    T, D, E, k = 600, 512, 16, 2
    S = T * k
    c = Gated(4, 24, 64, [9, 0, 33, 20], workloads.NVFP4, seed=18, T=31)
    w = 1.0 + normal(rng, D, scale=0.1)
    x, y, logits = normal(rng, T, D, dtype=torch.bfloat16), normal(rng, S, D), normal(rng, T, E)
    r, n = csf.route(logits, k), csf.rms_norm(x, w, x)
    dh = normal(rng, len(c.rows), c.F, dtype=torch.bfloat16)
    gu, dense, dg = c.forward(save=True)[1], c.dense(), normal(rng, T, k)
    calls = [
        (lambda v, **kw: csf.rms_norm(*v, **kw), (x, w, x)),
        (lambda v, **kw: csf.rms_norm(v[0], v[1], v[2], slots=v[3], gates=v[4], **kw), (y, w, x, r.slots, r.gates)),
        (lambda v, **kw: csf.rms_norm_backward(*v, **kw), (x, n.sum, w, n.rstd, x)),
        (lambda v, **kw: csf.route(*v, k, **kw), (logits,)),
        (lambda v, **kw: csf.combine_backward(*v, **kw), (x, y, r.slots, r.gates)),
        (lambda v, **kw: csf.route_backward(*v, **kw), (dg, logits, r.experts, r.gates)),
        (lambda v, **kw: csf.moe_gated(c.stack, *v, **kw), (c.tw, c.x, c.ta, c.te, c.tr)),
        (lambda v, **kw: csf.moe_gated_backward(c.stack, *v, **kw), (dense, c.tw, dh, gu, c.ta, c.te)),
    ]
    side = torch.cuda.Stream()
    busy = torch.empty(64 << 20, dtype=torch.float32, device=dev)

    def outputs(got):
        got = (got,) if isinstance(got, torch.Tensor) else got
        return [t for t in got if t is not None]

    for call, inputs in calls:
        want = outputs(call(inputs))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for i in range(20):  # a few milliseconds
                busy.fill_(float(i))
        copies = [t.clone() for t in inputs]
        sizes = [(t.shape, t.dtype) for t in copies]
        got = outputs(call(copies, stream=side))
        del copies
        junk = [torch.full(shape, 0x55, dtype=dtype, device=dev) for shape, dtype in sizes]
        side.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
        del junk


def test_bound_calls_captured_later_and_on_another_stream(dev):
    """Calls bound before a capture land in its graph; calls bound on a stream
    wait for the inputs that the current stream wrote since the last one."""
    rng = np.random.default_rng(23)
    T, E, k = 70, 6, 2
    c = Gated(E, 48, 256, [1] * E, workloads.NVFP4, seed=24)
    w = 1.0 + normal(rng, c.K, scale=0.1)
    x, logits = normal(rng, T, c.K, dtype=torch.bfloat16), normal(rng, T, E)

    def bind(**kw):
        norm = csf.bound(csf.rms_norm, x, w, x, **kw)
        route = csf.bound(csf.route, logits, k, **kw)
        n, r = norm(), route()
        return norm, route, csf.bound(csf.moe_gated, c.stack, c.tw, n.out, c.ta, r.expert_start, r.rows, **kw)

    def plain():
        n, r = csf.rms_norm(x, w, x), csf.route(logits, k)
        return n, r, csf.moe_gated(c.stack, c.tw, n.out, c.ta, r.expert_start, r.rows)

    def renew():
        x.copy_(normal(rng, T, c.K, dtype=torch.bfloat16))
        logits.copy_(normal(rng, T, E))

    def same(got, want):
        assert torch.equal(got[0].out, want[0].out) and torch.equal(got[0].sum, want[0].sum)
        assert all(torch.equal(a, b) for a, b in zip(got[1], want[1])) and torch.equal(got[2], want[2])

    calls = bind()
    [call() for call in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [call() for call in calls]
    for _ in range(4):
        renew()
        want = plain()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(out, want)
    side = torch.cuda.Stream()
    calls = bind(stream=side)
    big = torch.empty(64 << 20, dtype=torch.float32, device=dev)
    for _ in range(4):
        torch.cuda.current_stream().wait_stream(side)  # the last call has read its inputs
        for i in range(10):  # a few milliseconds before the inputs change
            big.fill_(float(i))
        renew()
        out = [call() for call in calls]
        torch.cuda.current_stream().wait_stream(side)
        same(out, plain())


def test_calls_on_the_default_stream_from_another(dev):
    """The default stream is no stream made here: it has no handle of its own."""
    rng = np.random.default_rng(29)
    x, w = normal(rng, 700, 2048, dtype=torch.bfloat16), torch.ones(2048, device=dev)
    want = csf.rms_norm(x, w, x)
    torch.cuda.synchronize()
    side, main = torch.cuda.Stream(), torch.cuda.default_stream()
    big = torch.empty(64 << 20, dtype=torch.float32, device=dev)
    with torch.cuda.stream(side):
        y = torch.zeros_like(x)
        call = csf.bound(csf.rms_norm, y, w, y)
        for i in range(10):
            big.fill_(float(i))
        y.copy_(x)
        got = csf.rms_norm(y, w, y, stream=main)  # waits for the copy
    assert torch.equal(got.out, want.out) and torch.equal(got.sum, want.sum)
    torch.cuda.synchronize()
    out = call().out  # bound under the side stream, called on the default one
    del call
    assert torch.equal(out, want.out)
