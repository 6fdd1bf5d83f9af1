"""fn_moe_swiglu: refusals on the CPU, parity with the oracle on the GPU, and a
run of the operators as a block uses them.

Tolerance, per element, with u = 2^-24.  The expert ids are those of the fp64
oracle exactly; the routing weights are fp64 values rounded once.  With
r = 1/rms (rounded to fp32: u), a dot product of K exact products of bf16
values in fp32 is off by at most e(K) = (8 + sqrt(K)) 2^-23 sum |terms|, as in
the projection's test.  So gate and up are off by e(d) r sum |x G| + 2 u |z|,
and an expert activation a = w silu(z_g) z_u by
    w (1.1 |z_u| dz_g + |silu(z_g)| dz_u) + 16 u |a|
(the slope of silu is at most 1.1; 16 u for its exponential, quotient and the
products), plus its rounding to bf16.  Those roundings are each within
2^-8 |a_i| and independent, so by Hoeffding's inequality their weighted sum
leaves 7 * 2^-8 (sum (a_i D_i)^2)^(1/2) with probability below 1e-10.  The
second product adds e(k I) sum |a D|, the residual u, the store 2^-8 |y|.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
import rmsnorm_linear_projection_flashnorm_b200 as fnb
from oracle import operators_oracle as P
from rmsnorm_linear_projection_flashnorm_b200 import torch_api as T

U = 2.0 ** -24
EPS = 1e-6
X, G, R, GU, WD, SB, RES, Y, IDS, W, WS = (i << 40 for i in range(1, 12))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fnb.build()
    fnb.lib()


# ------------------------------------------------------------------ CPU: refusals
def moe_(x=X, M=4, d=256, g=G, router=R, E=8, wgu=GU, wd=WD, I=128, k=2, score=0, sb=SB, renorm=1, scale=1.0, eps=EPS,
         res=RES, y=Y, ids=IDS, w=W, ws=WS, ws_bytes=1 << 30):
    return fnb.fn_moe_swiglu(x, M, d, g, router, E, wgu, wd, I, k, score, sb, renorm, scale, eps, res, y, ids, w, ws,
                             ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), fnb.FN_ERR_INVALID_ARG),
    (dict(d=0), fnb.FN_ERR_INVALID_ARG),
    (dict(E=0), fnb.FN_ERR_INVALID_ARG),
    (dict(I=0), fnb.FN_ERR_INVALID_ARG),
    (dict(k=0), fnb.FN_ERR_INVALID_ARG),
    (dict(k=9), fnb.FN_ERR_INVALID_ARG),                   # more than there are experts
    (dict(score=2), fnb.FN_ERR_INVALID_ARG),
    (dict(eps=-1.0), fnb.FN_ERR_INVALID_ARG),
    (dict(eps=math.nan), fnb.FN_ERR_INVALID_ARG),
    (dict(scale=math.inf), fnb.FN_ERR_INVALID_ARG),
    (dict(x=None), fnb.FN_ERR_INVALID_ARG),
    (dict(router=None), fnb.FN_ERR_INVALID_ARG),
    (dict(wgu=None), fnb.FN_ERR_INVALID_ARG),
    (dict(wd=None), fnb.FN_ERR_INVALID_ARG),
    (dict(y=None), fnb.FN_ERR_INVALID_ARG),
    (dict(ws=None), fnb.FN_ERR_WORKSPACE),
    (dict(M=65), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(d=96), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(I=192), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(E=513), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(E=64, k=17), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(E=512, d=1 << 22), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(E=512, I=1 << 22), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(x=X + 8), fnb.FN_ERR_ALIGNMENT),
    (dict(g=G + 4), fnb.FN_ERR_ALIGNMENT),
    (dict(router=R + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(wgu=GU + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(wd=WD + 8), fnb.FN_ERR_ALIGNMENT),
    (dict(sb=SB + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(res=RES + 1), fnb.FN_ERR_ALIGNMENT),
    (dict(y=Y + 1), fnb.FN_ERR_ALIGNMENT),
    (dict(ids=IDS + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(w=W + 1), fnb.FN_ERR_ALIGNMENT),
    (dict(ws=WS + 8), fnb.FN_ERR_ALIGNMENT),
    (dict(y=X + 64), fnb.FN_ERR_ALIAS),                    # not in place
    (dict(y=RES + 64), fnb.FN_ERR_ALIAS),
    (dict(y=GU + 64), fnb.FN_ERR_ALIAS),
    (dict(y=WD + 64), fnb.FN_ERR_ALIAS),
    (dict(y=R + 64), fnb.FN_ERR_ALIAS),
    (dict(ids=X + 4), fnb.FN_ERR_ALIAS),
    (dict(w=IDS + 4), fnb.FN_ERR_ALIAS),
    (dict(ids=Y + 4), fnb.FN_ERR_ALIAS),
    (dict(ws=Y - 1024), fnb.FN_ERR_ALIAS),
    (dict(ws=SB - 512), fnb.FN_ERR_ALIAS),
])
def test_refusals(kw, code):
    assert moe_(**kw) == code


def test_empty_batch_and_workspace_size():
    assert moe_(M=0, x=None, router=None, wgu=None, wd=None, y=None, ws=None) == fnb.FN_OK
    assert fnb.fn_workspace_size_moe(0, 64, 128, 8, 2) == 256
    assert fnb.fn_workspace_size_moe(65, 64, 128, 8, 2) == 256
    a, b = (fnb.fn_workspace_size_moe(16, 2048, 1024, 64, k) for k in (1, 8))
    assert b - a == (64 - 16) * 16 * 1024 * 2              # min(E, M k) experts' activations


def test_torch_api_refuses_what_the_library_cannot_see():
    bf = torch.bfloat16
    x, r = torch.zeros(2, 64, dtype=bf), torch.zeros(4, 64, dtype=bf)
    gu, wd, g = torch.zeros(4, 64, 256, dtype=bf), torch.zeros(4, 128, 64, dtype=bf), torch.ones(64)
    for bad in (lambda: T.moe_swiglu(x, g, r, gu, wd, 2, EPS),                       # not on a GPU
                lambda: T.moe_swiglu(x.float(), g, r, gu, wd, 2, EPS),
                lambda: T.moe_swiglu(x, g[:32], r, gu, wd, 2, EPS),
                lambda: T.moe_swiglu(x, g, r[:3], gu, wd, 2, EPS),
                lambda: T.moe_swiglu(x, g, r, gu[:, :, :128], wd, 2, EPS),
                lambda: T.moe_swiglu(x, g, r, gu, wd.transpose(1, 2), 2, EPS),
                lambda: T.moe_swiglu(x, g, r, gu, wd, 5, EPS),
                lambda: T.moe_swiglu(x, g, r, gu, wd, 2, EPS, score="top"),
                lambda: T.moe_swiglu(x, g, r, gu, wd, 2, EPS, select_bias=torch.zeros(3)),
                lambda: T.moe_swiglu(x, g, r, gu, wd, 2, EPS, residual=x[:1]),
                lambda: T.fold_experts(gu, g, gu[:, :, :128])):
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------------ GPU: parity
class Layer:
    """Random weights of one layer on the GPU and the 64-bit values they hold."""

    def __init__(self, d, I, E, seed, gain=True):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()
        self.d, self.I, self.E = d, I, E
        self.g = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")) if gain else None
        self.router = rnd(E, d, std=2 * d ** -0.5)
        self.gate, self.up = rnd(E, d, I, std=d ** -0.5), rnd(E, d, I, std=d ** -0.5)
        self.down = rnd(E, I, d, std=2 * I ** -0.5)
        ones = torch.ones(d, device="cuda")
        self.Wgu = T.fold_experts(self.gate, self.g if gain else ones, self.up)
        self.bias = torch.randn(E, generator=g, device="cuda") * 0.3

    def x(self, M, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        s = torch.exp(torch.randn(M, 1, generator=g, device="cuda"))
        return (torch.randn(M, self.d, generator=g, device="cuda") * s).bfloat16()

    def reference(self, x, k, residual=None, **route):
        """(y, its tolerance, ids, weights) from the oracle's route, the stored
        (folded) weights and the formulas above, in 64 bits."""
        gain = np.ones(self.d) if self.g is None else self.g.cpu().numpy()
        sb = route.pop("select_bias", None)
        ids, w = P.moe_route(x.cpu(), gain, self.router.cpu(), k, EPS,
                             select_bias=None if sb is None else sb.cpu().numpy(), **route)
        M, d, I = x.shape[0], self.d, self.I
        xd = x.double()
        r = torch.rsqrt(xd.square().mean(1, keepdim=True) + EPS)

        def e(K):
            return (8 + math.sqrt(K)) * 2 * U
        y = torch.zeros_like(xd) if residual is None else residual.double().clone()
        lin, mag, sq = torch.zeros_like(xd), torch.zeros_like(xd), torch.zeros_like(xd)
        for ex in range(self.E):
            rows, slot = np.nonzero(ids == ex)
            if not rows.size:
                continue
            rt, wt = torch.from_numpy(rows).cuda(), torch.from_numpy(w[rows, slot]).cuda()[:, None]
            gu = self.Wgu[ex].double().view(d, I // 128, 2, 128)
            G_, U_ = gu[:, :, 0].reshape(d, I), gu[:, :, 1].reshape(d, I)
            h = r[rt] * xd[rt]
            zg, zu = h @ G_, h @ U_
            dg = e(d) * (h.abs() @ G_.abs()) + 2 * U * zg.abs()
            du = e(d) * (h.abs() @ U_.abs()) + 2 * U * zu.abs()
            s = zg * torch.sigmoid(zg)
            a = wt * s * zu
            da = wt.abs() * (1.1 * zu.abs() * dg + s.abs() * du) + 16 * U * a.abs()
            D = self.down[ex].double()
            y[rt] += a @ D
            lin[rt] += da @ D.abs()
            mag[rt] += a.abs() @ D.abs()
            sq[rt] += a.square() @ D.square()
        tol = lin + e(k * I) * mag + 7 * 2 ** -8 * sq.sqrt() * (1 + 2 ** -7) + U * y.abs()
        tol += 2 ** -8 * y.abs() * (1 + 2 ** -7) + 1e-30
        if residual is not None:
            tol += U * residual.double().abs()
        return y, tol, ids, w


def check(layer, M, k, seed=0, residual=True, ws=None, x=None, alias=False, **route):
    x = layer.x(M, seed) if x is None else x
    res = None if not residual else x.clone() if alias else layer.x(M, seed + 1)
    ref, tol, ids, w = layer.reference(x, k, res, **route)
    buf = torch.full((M + 2, layer.d), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:M + 1]
    if alias:
        out.copy_(x)
        x = res = out
    y, gi, gw = T.moe_swiglu(x, layer.g, layer.router, layer.Wgu, layer.down, k, EPS, residual=res, ws=ws, out=out,
                             **route)
    torch.cuda.synchronize()
    assert y is out and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert np.array_equal(gi.cpu().numpy(), ids)
    assert np.allclose(gw.double().cpu().numpy(), w, rtol=2 * U, atol=1e-37)
    over = (y.double() - ref).abs() - tol
    assert not torch.isnan(y).any() and over.max() <= 0, over.max()
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 13, 16, 17, 19, 32, 33, 37, 64])
@pytest.mark.parametrize("d,I,E,k", [(256, 128, 8, 2), (64, 128, 3, 1), (320, 256, 40, 7)])
def test_rows(M, d, I, E, k):
    check(Layer(d, I, E, seed=d), M, k, seed=M)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_routing(score, biased, renorm):
    layer = Layer(512, 128, 33, seed=1)
    for M, k in ((5, 3), (40, 16)):
        check(layer, M, k, score=score, select_bias=layer.bias if biased else None, renorm=renorm, route_scale=2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("M,d,I,E,k", [(1, 2048, 1024, 64, 8), (13, 2048, 768, 128, 8), (64, 4096, 2048, 8, 2),
                                       (64, 1024, 128, 512, 16), (7, 64, 4096, 2, 2), (3, 8192, 128, 1, 1),
                                       (24, 128, 128, 300, 5), (64, 1088, 640, 100, 6)])
def test_sizes(M, d, I, E, k):
    check(Layer(d, I, E, seed=M + E), M, k, residual=M != 7)


@pytest.mark.gpu
def test_without_gain_and_in_place():
    layer = Layer(384, 256, 12, seed=3, gain=False)
    for M in (1, 20, 64):
        check(layer, M, 4)
        check(layer, M, 4, alias=True)


@pytest.mark.gpu
def test_ties_go_to_the_lower_expert():
    """Router rows of small integers: the logits are sums without rounding."""
    layer = Layer(256, 128, 20, seed=4, gain=False)
    g = torch.Generator().manual_seed(1)
    layer.router.copy_(torch.randint(-1, 2, (20, 256), generator=g).bfloat16())
    layer.router[7] = layer.router[3]
    layer.router[19] = layer.router[3]
    layer.router[10:14] = layer.router[2]
    x = torch.randint(-2, 3, (9, 256), generator=g).bfloat16().cuda()
    x[0] = 0                                                # every logit alike
    check(layer, 9, 6, x=x)
    check(layer, 9, 6, x=x, score="sigmoid", select_bias=torch.zeros(20, device="cuda"))


@pytest.mark.gpu
def test_experts_masked_by_the_selection_bias():
    """A bias of the lowest value or minus infinity takes experts out as long
    as others are left; then the lower indices fill up."""
    layer = Layer(256, 128, 10, seed=5)
    for low in (-math.inf, torch.finfo(torch.float32).min):
        sb = torch.full((10,), low, device="cuda")
        sb[torch.tensor([2, 5, 6])] = 0
        check(layer, 6, 3, select_bias=sb)
        check(layer, 6, 5, select_bias=torch.where(sb == 0, sb, -math.inf))


@pytest.mark.gpu
def test_values_far_apart():
    """Rows of zeros, of tiny and of huge activations; a softmax that leaves
    one expert; sigmoids that underflow in 32 bits."""
    layer = Layer(256, 128, 16, seed=6)
    x = layer.x(6, 1)
    x[1] = 0
    x[2] *= 1e-18
    x[3] *= 1e17
    layer.router *= 8
    check(layer, 6, 4, x=x, residual=False)
    check(layer, 6, 4, x=x, residual=False, renorm=False)
    check(layer, 6, 4, x=x, residual=False, renorm=False, score="sigmoid")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 40])
def test_non_finite_rows_stay_in_their_rows(M):
    layer = Layer(256, 128, 8, seed=7)
    x = layer.x(M, 2)

    def call(x):
        y, ids, w = T.moe_swiglu(x, layer.g, layer.router, layer.Wgu, layer.down, 3, EPS)
        torch.cuda.synchronize()
        return y, ids, w
    clean, cid, _ = call(x)
    x[1, 5], x[3, 7] = math.nan, math.inf
    y, ids, w = call(x)
    for m in (1, 3):
        assert torch.isnan(y[m]).all() and torch.isnan(w[m]).all()
        assert ids[m].tolist() == [0, 1, 2]                 # no key is a number
    keep = [i for i in range(M) if i not in (1, 3)]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(ids[keep], cid[keep])


@pytest.mark.gpu
def test_repeats_capture_and_streams():
    layer = Layer(1024, 384, 32, seed=8)
    ws = T.Workspace("cuda")

    def call(x, ws, out=None, stream=None):
        return T.moe_swiglu(x, layer.g, layer.router, layer.Wgu, layer.down, 4, EPS, residual=x, ws=ws, out=out,
                            stream=stream)[0]
    x = layer.x(11, 1)
    check(layer, 11, 4, x=x, residual=False)
    ref = call(x, ws)
    torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(call(x, ws), ref)
    # captured: two layers in a row through one workspace
    out = torch.empty_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, ws, out=out)
        call(out, ws, out=out)
    x.copy_(layer.x(11, 9))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    a = call(x, ws)
    b = call(a, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, b)
    # two calls at once, each with its own workspace, and workspaces made on the call's stream
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [T.Workspace("cuda"), None]
    torch.cuda.synchronize()
    outs = [call(x, wss[j], stream=s[j]) for _ in range(8) for j in range(2)]
    raw = call(x, None, stream=s[0].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for o in outs + [raw])


@pytest.mark.gpu
def test_timeout_is_reported():
    """A commit that never comes: the epilogue's wait runs out, the call ends
    and the status word says so."""
    layer = Layer(256, 128, 8, seed=9)
    x, ws = layer.x(4, 1), T.Workspace("cuda")
    fnb.fn_set_debug(fnb.FN_DEBUG_WAIT_BUDGET_NS, 20_000_000)
    fnb.fn_set_debug(fnb.FN_DEBUG_WITHHOLD_ARRIVE, 1)
    try:
        T.moe_swiglu(x, layer.g, layer.router, layer.Wgu, layer.down, 2, EPS, ws=ws)
        torch.cuda.synchronize()
        assert ws.status()[0] == fnb.FN_ERR_TIMEOUT
    finally:
        fnb.fn_set_debug(fnb.FN_DEBUG_WITHHOLD_ARRIVE, 0)
        fnb.fn_set_debug(fnb.FN_DEBUG_WAIT_BUDGET_NS, 2_000_000_000)
    ws.buf.zero_()
    check(layer, 4, 2, ws=ws)
    assert ws.status()[0] == fnb.FN_OK


@pytest.mark.gpu
def test_decode_step_of_a_block_through_one_workspace():
    """norm_proj -> proj (+ residual) -> moe_swiglu (+ residual) -> norm_proj
    (head) -> token_logprobs, each step against the oracle on its own inputs;
    the counters of every kernel that shares the workspace end at zero."""
    d, V, M = 512, 1280, 9
    layer = Layer(d, 256, 16, seed=10)
    g = torch.Generator(device="cuda").manual_seed(2)
    Wv = (torch.randn(d, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    Wo = (torch.randn(d, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    Wh = (torch.randn(d, V, generator=g, device="cuda") * d ** -0.5).bfloat16()
    gain = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    Wvf, _ = T.fold(Wv, gain)
    Whf, _ = T.fold(Wh, gain)
    ws = T.Workspace("cuda")
    x = layer.x(M, 5)
    v = T.norm_proj(x, Wvf, d, EPS, ws=ws)
    h = T.proj(v, Wo, residual=x, ws=ws)
    y, _, _ = T.moe_swiglu(h, layer.g, layer.router, layer.Wgu, layer.down, 4, EPS, residual=h, ws=ws)
    logits = T.norm_proj(y, Whf, V, EPS, ws=ws)
    t = torch.arange(M, device="cuda", dtype=torch.int32) * 97
    lp = T.token_logprobs(logits, t, top_k=5)
    torch.cuda.synchronize()
    assert ws.status()[0] == fnb.FN_OK and (ws.buf[:256] == 0).all()
    ones = np.ones(d)

    def close(a, b, tol):
        a = a.double().cpu().numpy()
        assert np.max(np.abs(a - b) / (1 + np.abs(b))) <= tol
    close(v, O.norm_proj(x.cpu(), ones, Wvf.double().cpu().numpy(), EPS), 2 ** -7)
    close(h, P.project(v.cpu(), Wo.cpu(), residual=x.cpu()), 2 ** -7)
    ref, tol, _, _ = layer.reference(h, 4, h)
    assert ((y.double() - ref).abs() <= tol).all()
    close(logits, O.norm_proj(y.cpu(), ones, Whf.double().cpu().numpy(), EPS), 2 ** -7)
    elp, eH, _, eids, _ = P.token_logprobs(logits.cpu(), t.cpu(), 5)
    close(lp.logprob, elp, 1e-5)
    close(lp.entropy, eH, 1e-5)
    assert np.array_equal(lp.top_ids.cpu().numpy(), eids)


@pytest.mark.gpu
def test_weights_past_32_bits():
    """Experts whose weights lie past 2^31 elements."""
    d, I, E = 4096, 4096, 72                                # 72 x 4096 x 8192 elements of gate/up
    layer = Layer.__new__(Layer)
    layer.d, layer.I, layer.E, layer.g = d, I, E, None
    g = torch.Generator(device="cuda").manual_seed(3)
    layer.router = (torch.randn(E, d, generator=g, device="cuda") * d ** -0.5).bfloat16()
    layer.Wgu = torch.empty(E, d, 2 * I, dtype=torch.bfloat16, device="cuda")
    layer.down = torch.empty(E, I, d, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        layer.Wgu[e] = torch.randn(d, 2 * I, generator=g, device="cuda", dtype=torch.bfloat16) * d ** -0.5
        layer.down[e] = torch.randn(I, d, generator=g, device="cuda", dtype=torch.bfloat16) * 2 * I ** -0.5
    sb = torch.zeros(E, device="cuda")
    sb[torch.tensor([0, 68, 70, 71])] = 10.0                # the first and the last experts
    for M in (1, 20):
        check(layer, M, 4, select_bias=sb)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [17, 32, 33, 55, 64])
@pytest.mark.parametrize("d,I,E,k", [(4544, 384, 5, 4), (64, 6912, 3, 2), (192, 2176, 16, 8), (1536, 512, 4, 1), (5120, 128, 1, 1)])
def test_shared_tiles_of_many_rows(M, d, I, E, k):
    """Few tiles with long k ranges: every tile of both products is shared by
    many CTAs, and fix-up kernels finish them."""
    layer = Layer(d, I, E, seed=d + E)
    ws = T.Workspace("cuda")
    check(layer, M, k, seed=M, ws=ws)
    check(layer, M, k, seed=M + 1, ws=ws, alias=True)
    assert ws.status()[0] == fnb.FN_OK and (ws.buf[:256] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 20, 64])
def test_norms_of_the_whole_range(M):
    """Activations whose squares leave the range of 32 bits.  Without eps the
    layer does not depend on the scale of its rows, and a power of two changes
    no rounding: the same experts, weights and outputs, bit by bit."""
    layer = Layer(256, 128, 16, seed=11)
    x = layer.x(M, 3)

    def call(x):
        out = T.moe_swiglu(x, layer.g, layer.router, layer.Wgu, layer.down, 4, 0.0)
        torch.cuda.synchronize()
        return out
    y, ids, w = call(x)
    ref_ids, ref_w = P.moe_route(x.cpu(), layer.g.cpu().numpy(), layer.router.cpu(), 4, 0.0)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    assert np.allclose(w.double().cpu().numpy(), ref_w, rtol=2 * U, atol=1e-37)
    for e in (83, 100, -66, -83):
        a, b, c = call(x * 2.0 ** e)
        assert torch.equal(b, ids) and torch.equal(c, w) and torch.equal(a, y), e
    big = x.clone()
    big[1] *= 2.0 ** 83
    check(layer, M, 4, x=big, residual=False)
