"""fn_proj: refusals on the CPU, parity with the oracle on the GPU.

Tolerance, per element, with u = 2^-24: products of bf16 values are exact in
fp32; the tensor cores and the partial sums add K of them in fp32, so the sum
is off by at most K u sum |x W| in the worst order, and by a small multiple of
sqrt(K) u (sum of squares)^(1/2) in practice: the bound used is
(8 + sqrt(K)) 2^-23 * sum_k |x_k W_k| (truncating adders: 2 u per add), times
the activation's slope, at most 1.2.  The activation itself carries 16 u of
its value (ex2-based exponentials, erfc), of |z| for the tanh form's argument
(its exponential's relative error is the argument's absolute one, 2 u |u2|,
damped by the logistic factor).  The bias and residual add u each, and the
store eps / 2 of the value.
"""
import math
import weakref

import numpy as np
import pytest
import torch

import oracle as O
import rmsnorm_linear_projection_flashnorm_b200 as fnb
from rmsnorm_linear_projection_flashnorm_b200 import torch_api as T

U = 2.0 ** -24
X, W, Y, R, B, WS = 1 << 30, 1 << 34, 1 << 36, 1 << 37, 1 << 38, 1 << 39


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fnb.build()
    fnb.lib()


# ------------------------------------------------------------------ CPU: refusals
def proj_(x=X, ldx=256, M=4, K=256, w=W, ldw=512, N=512, bias=B, act=0, res=R, ldr=512, dt=0, y=Y, ldy=512, ws=WS,
          ws_bytes=1 << 30):
    return fnb.fn_proj(x, ldx, M, K, w, ldw, N, bias, act, res, ldr, dt, y, ldy, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), fnb.FN_ERR_INVALID_ARG),
    (dict(K=0), fnb.FN_ERR_INVALID_ARG),
    (dict(N=0), fnb.FN_ERR_INVALID_ARG),
    (dict(ldx=248), fnb.FN_ERR_INVALID_ARG),
    (dict(ldw=504), fnb.FN_ERR_INVALID_ARG),
    (dict(ldy=511), fnb.FN_ERR_INVALID_ARG),
    (dict(ldr=511), fnb.FN_ERR_INVALID_ARG),
    (dict(act=5), fnb.FN_ERR_INVALID_ARG),
    (dict(act=-1), fnb.FN_ERR_INVALID_ARG),
    (dict(dt=1), fnb.FN_ERR_INVALID_ARG),                  # fp16 output
    (dict(x=None), fnb.FN_ERR_INVALID_ARG),
    (dict(w=None), fnb.FN_ERR_INVALID_ARG),
    (dict(y=None), fnb.FN_ERR_INVALID_ARG),
    (dict(ws=None), fnb.FN_ERR_WORKSPACE),
    (dict(ldx=260), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(ldw=513), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(M=(1 << 30) + 1), fnb.FN_ERR_UNSUPPORTED_SHAPE),
    (dict(x=X + 8), fnb.FN_ERR_ALIGNMENT),
    (dict(w=W + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(y=Y + 1), fnb.FN_ERR_ALIGNMENT),
    (dict(dt=2, y=Y + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(dt=2, res=R + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(bias=B + 2), fnb.FN_ERR_ALIGNMENT),
    (dict(ws=WS + 8), fnb.FN_ERR_ALIGNMENT),
    (dict(y=X + 64), fnb.FN_ERR_ALIAS),
    (dict(y=W + 64), fnb.FN_ERR_ALIAS),
    (dict(y=R + 2), fnb.FN_ERR_ALIAS),                     # overlaps the residual, not in place
    (dict(y=R, ldy=520), fnb.FN_ERR_ALIAS),                # in place with another row stride
    (dict(y=B + 16), fnb.FN_ERR_ALIAS),
    (dict(y=WS + 512), fnb.FN_ERR_ALIAS),
    (dict(ws=R + 1024), fnb.FN_ERR_ALIAS),
])
def test_refusals(kw, code):
    assert proj_(**kw) == code


def test_empty_batch_and_workspace_size():
    assert proj_(M=0, x=None, w=None, y=None, ws=None) == fnb.FN_OK
    assert fnb.fn_workspace_size_proj(0, 64, 64) == 256
    sizes = [fnb.fn_workspace_size_proj(m, 4096, 4096) for m in (1, 16, 17, 32, 33, 64)]
    assert sizes[0] == sizes[1] < sizes[2] == sizes[3] < sizes[4] == sizes[5]


def test_torch_api_refuses_what_the_library_cannot_see():
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    for bad in (lambda: T.proj(x, w), lambda: T.proj(x.float(), w), lambda: T.proj(x, w[:7]), lambda: T.proj(x, w.t()),
                lambda: T.proj(x, w, act="tanh"), lambda: T.proj(x, w, bias=torch.zeros(15)),
                lambda: T.proj(x, w, residual=torch.zeros(2, 15)),
                lambda: T.proj(x, w, residual=torch.zeros(2, 16), out=torch.zeros(2, 16, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------------ GPU: parity
def padded(rows, cols, ld, seed, std=1.0):
    """bf16 [rows, cols] in rows of ld; what lies between the rows is NaN."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((rows, ld), math.nan, dtype=torch.bfloat16)
    buf[:, :cols] = (torch.randn(rows, cols, generator=g) * std).bfloat16()
    return buf.cuda()[:, :cols]


def up8(n):
    return (n + 7) // 8 * 8


def case(M, K, N, bias=False, act="none", residual=False, fp32=False, pad=0, seed=0, ws=None, alias=False):
    x = padded(M, K, up8(K) + pad, seed)
    w = padded(K, N, up8(N) + pad, seed + 1, K ** -0.5)
    g = torch.Generator().manual_seed(seed + 2)
    b = torch.randn(N, generator=g).cuda() if bias else None
    dt = torch.float32 if fp32 else torch.bfloat16
    r = torch.randn(M, N + 3, generator=g).to(dt).cuda()[:, 1:N + 1] if residual else None
    buf = torch.full((M + 2, N + 5), 7.0, dtype=dt, device="cuda")
    out = buf[1:M + 1, 2:N + 2]
    rc = None if r is None else r.clone()
    if alias:
        out.copy_(r)
        r = out
    y = T.proj(x, w, bias=b, act=act, residual=r, ws=ws, out=out)
    torch.cuda.synchronize()
    assert y is out
    buf[1:M + 1, 2:N + 2], got = 7.0, y.double().cpu().numpy()
    assert (buf == 7).all(), "wrote outside the output"
    xd, wd = x.double().cpu().numpy(), w.double().cpu().numpy()
    ref = O.project(xd, wd, None if b is None else b.cpu().numpy(), act, None if rc is None else rc.double().cpu())
    mag = np.abs(xd) @ np.abs(wd)
    z = np.abs(O.project(xd, wd, None if b is None else b.cpu().numpy()))
    tol = 1.2 * ((8 + math.sqrt(K)) * 2 * U * mag + U * z) + 16 * U * z * (1 + (z if act == "gelu_tanh" else 0))
    if residual:
        tol = tol + U * (np.abs(ref) + np.abs(rc.double().cpu().numpy()))
    tol = tol + torch.finfo(dt).eps / 2 * np.abs(ref) * (1 + 2 ** -7) + 1e-30
    bad = np.abs(got - ref) - tol
    assert not np.isnan(got).any() and bad.max() <= 0, (bad.max(), np.unravel_index(bad.argmax(), bad.shape))


MS = [1, 2, 15, 16, 17, 31, 33, 64, 65, 96, 97, 129, 256, 257, 300, 513]


@pytest.mark.gpu
@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("K,N", [(64, 128), (1, 1), (7, 3), (200, 130), (1000, 257), (4096, 72)])
def test_sizes(M, K, N):
    case(M, K, N, residual=True, bias=True, seed=M + K)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("fp32", [False, True])
def test_activations(M, act, fp32):
    case(M, 333, 259, bias=True, act=act, residual=False, fp32=fp32, pad=8, seed=5)
    case(M, 333, 259, bias=True, act=act, residual=True, fp32=fp32, pad=16, seed=6)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (16, 2048, 4096), (64, 4096, 2048), (45, 2051, 4099),
                                   (8, 16384, 100), (64, 16000, 640), (3, 64, 30000), (1, 14336, 4096)])
def test_few_rows_split_k(M, K, N):
    case(M, K, N, residual=True, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(300, 14336, 1024), (65, 8192, 4096), (128, 16384, 256), (1000, 4096, 2048),
                                   (4096, 512, 1024), (700, 2000, 6144), (2048, 4096, 2560), (257, 1024, 20000)])
def test_many_rows(M, K, N):
    case(M, K, N, residual=True, bias=True, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 64, 200])
@pytest.mark.parametrize("fp32", [False, True])
def test_residual_in_place(M, fp32):
    case(M, 1024, 520, residual=True, fp32=fp32, seed=3, alias=True)


@pytest.mark.gpu
def test_one_workspace_for_every_call_in_turn():
    """Calls of other sizes and of the fused projections in between leave the
    counters of the shared tiles at zero."""
    import workloads as WL
    ws = T.Workspace("cuda")
    inp = WL.case(8, 512, 1024, False, seed=3)
    Wp, _ = T.fold(inp["W"].cuda(), inp["g"].cuda())
    for i, (M, K, N) in enumerate([(1, 4096, 512), (300, 8192, 512), (40, 1000, 3000), (1, 4096, 512), (300, 8192, 512)]):
        case(M, K, N, seed=i, ws=ws)
        T.norm_proj(inp["x"].cuda(), Wp, 1024, 1e-6, ws=ws)
    assert ws.status()[0] == fnb.FN_OK
    assert (ws.buf[:256] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(7, 4096, 1000), (200, 8192, 1024)])
def test_repeats_capture_and_streams(M, K, N):
    x, w = padded(M, K, up8(K), 1), padded(K, N, up8(N), 2, K ** -0.5)
    ws = T.Workspace("cuda")
    ref = T.proj(x, w, ws=ws)
    torch.cuda.synchronize()
    for _ in range(5):
        y = T.proj(x, w, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    out = torch.empty_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.proj(x, w, ws=ws, out=out)
        T.proj(x, w, ws=ws, out=out, residual=out)
    x.copy_(padded(M, K, up8(K), 9))
    g.replay()
    torch.cuda.synchronize()
    a = T.proj(x, w, ws=ws)
    b = T.proj(x, w, ws=ws, residual=a)
    torch.cuda.synchronize()
    assert torch.equal(out, b)
    # two calls at once, each with its own workspace
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [T.Workspace("cuda") for _ in s]
    for q in wss:
        q.reserve(fnb.fn_workspace_size_proj(M, K, N))
    outs = [[torch.empty_like(ref) for _ in range(8)] for _ in s]
    torch.cuda.synchronize()
    for i in range(8):
        for j in range(2):
            T.proj(x, w, ws=wss[j], out=outs[j][i], stream=s[j])
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for os_ in outs for o in os_)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 100])
def test_non_finite_rows_stay_in_their_rows(M):
    x, w = padded(M, 512, 512, 1), padded(512, 384, 384, 2)
    clean = T.proj(x, w)
    x[1, 5], x[2, 7] = math.nan, math.inf
    y = T.proj(x, w)
    torch.cuda.synchronize()
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 100])
def test_timeout_is_reported(M):
    """A commit that never comes: the epilogue's wait runs out, the call ends
    and the status word says so."""
    x, w = padded(M, 512, 512, 1), padded(512, 384, 384, 2)
    ws = T.Workspace("cuda")
    fnb.fn_set_debug(fnb.FN_DEBUG_WAIT_BUDGET_NS, 20_000_000)
    fnb.fn_set_debug(fnb.FN_DEBUG_WITHHOLD_ARRIVE, 1)
    try:
        T.proj(x, w, ws=ws)
        torch.cuda.synchronize()
        assert ws.status()[0] == fnb.FN_ERR_TIMEOUT
    finally:
        fnb.fn_set_debug(fnb.FN_DEBUG_WITHHOLD_ARRIVE, 0)
        fnb.fn_set_debug(fnb.FN_DEBUG_WAIT_BUDGET_NS, 2_000_000_000)
    ws.buf.zero_()
    y = T.proj(x, w, ws=ws)
    torch.cuda.synchronize()
    assert ws.status()[0] == fnb.FN_OK and torch.isfinite(y).all()


def aligned(M, K, N, fp32, residual, act, seed):
    """Contiguous output and residual: the epilogue's vector form where N is a
    multiple of 4.  What the tolerance counts is in the module's docstring."""
    x, w = padded(M, K, up8(K), seed), padded(K, N, up8(N), seed + 1, K ** -0.5)
    g = torch.Generator().manual_seed(seed + 2)
    b = torch.randn(N, generator=g).cuda()
    dt = torch.float32 if fp32 else torch.bfloat16
    r = torch.randn(M, N, generator=g).to(dt).cuda() if residual else None
    y = T.proj(x, w, bias=b, act=act, residual=r, out_dtype=dt)
    torch.cuda.synchronize()
    xd, wd = x.double(), w.double()
    z = xd @ wd + b.double()
    ref = z * torch.sigmoid(z) if act == "silu" else z
    if residual:
        ref = ref + r.double()
    tol = 1.2 * ((8 + math.sqrt(K)) * 2 * U * (xd.abs() @ wd.abs()) + U * z.abs()) + 16 * U * z.abs()
    tol = tol + U * ref.abs() + (U * r.double().abs() if residual else 0)
    tol = tol + torch.finfo(dt).eps / 2 * ref.abs() * (1 + 2 ** -7) + 1e-30
    over = (y.double() - ref).abs() - tol
    assert not torch.isnan(y).any() and over.max() <= 0, over.max()


@pytest.mark.gpu
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K,N", [(65, 200, 128), (100, 512, 260), (257, 333, 1000), (300, 14336, 1024), (512, 16384, 512),
                                   (1000, 256, 4100), (4099, 128, 516), (700, 8192, 2052)])
def test_aligned_output(M, K, N, fp32, residual):
    aligned(M, K, N, fp32, residual, "silu" if M == 257 else "none", seed=M + N)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(5, 64, 1 << 16), (64, 128, 1 << 15)])
def test_aligned_output_few_rows(M, K, N):
    aligned(M, K, N, False, True, "none", seed=1)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Output, residual (in place) and weight rows whose element offsets pass
    2^31: the last rows and columns are right, and the first are not theirs."""
    M, K, N = 66000, 64, 33000
    x, w = padded(M, K, K, 1), padded(K, N, N, 2, K ** -0.5)
    y = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    T.proj(x, w, residual=y, out=y)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 255, 256, M // 2, M - 257, M - 2, M - 1], device="cuda")
    ref = x[rows].double() @ w.double() + 1
    tol = 2 ** -8 * ref.abs() * (1 + 2 ** -7) + (8 + math.sqrt(K)) * 2 * U * (x[rows].double().abs() @ w.double().abs()) + 4 * U
    assert ((y[rows].double() - ref).abs() <= tol).all()
    del y
    # a weight of more than 2^31 elements under few rows
    K, N = 70000, 32768
    x, w = padded(3, K, K, 3), torch.zeros(K, N, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 65535, 65536, K - 2, K - 1], device="cuda")
    w[at] = (torch.randn(len(at), N, device="cuda") * 0.5).bfloat16()
    y = T.proj(x, w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    ref = x[:, at].double() @ w[at].double()
    mag = x[:, at].double().abs() @ w[at].double().abs()
    assert ((y.double() - ref).abs() <= (8 + math.sqrt(K)) * 2 * U * mag + U * ref.abs() + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(16, 256, 38000), (16, 256, 38016), (64, 64, 28416), (48, 128, 30001), (64, 6144, 28416),
                                   (128, 1024, 9472), (128, 1024, 9600), (65, 4096, 1000), (120, 100, 72), (20, 64, 16384)])
def test_few_rows_many_columns(M, K, N):
    """Both sides of the choice between the weight-stream and the tile kernel,
    whole tiles and shared ones, rows on and off the 128-byte lines."""
    case(M, K, N, residual=True, bias=True, seed=M)
    aligned(M, K, N, False, True, "none", seed=K)
    aligned(M, K, N, True, False, "silu", seed=K)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(3737, 75, 110), (2671, 151, 29), (498, 416, 277), (590, 64, 64), (1000, 512, 512), (130, 1024, 260)])
@pytest.mark.parametrize("fp32", [False, True])
def test_small_tiles(M, K, N, fp32):
    """Few tiles and a short k range: fewer rows to a tile."""
    case(M, K, N, residual=True, bias=True, act="gelu", fp32=fp32, seed=M)
    aligned(M, K, N, fp32, True, "silu", seed=N)


def test_workspace_keeps_the_buffers_it_replaced():
    """A captured graph holds the address of the buffer it was captured with."""
    ws = T.Workspace("cpu")
    refs = [weakref.ref(ws.buf)]
    for need in (1000, 1100, 5000, 100, 5000, 1 << 20):
        buf = ws.reserve(need)
        assert buf is ws.buf and buf.numel() >= need and not buf.any()
        if refs[-1]() is not buf:
            refs.append(weakref.ref(buf))
        buf.fill_(1)
        del buf
        ws.buf.zero_()
    bufs = [r() for r in refs]
    assert len(bufs) == 5 and all(b is not None for b in bufs)
    assert sum(b.numel() for b in bufs) < 2 * ws.buf.numel()


def test_workspace_does_not_grow_in_a_capture(monkeypatch):
    """Its zeroing would only be recorded, and the memory would be the graph's."""
    ws = T.Workspace("cpu")
    ws.reserve(1000)
    own = ws.buf
    monkeypatch.setattr(T, "_capturing", lambda device: True, raising=False)
    assert ws.reserve(900) is own
    a, b = ws.reserve(2000), ws.reserve(2000)
    assert a.numel() == b.numel() == 2000 and not a.any() and a is not b and ws.buf is own


@pytest.mark.gpu
def test_workspace_grows_behind_a_captured_graph():
    x, w = padded(7, 4096, 4096, 1), padded(4096, 1000, 1000, 2, 1 / 64)
    xl, wl = padded(100, 8192, 8192, 3), padded(8192, 512, 512, 4, 1 / 90)      # needs 19 MB where the first needs 2
    ws = T.Workspace("cuda")
    ref, large = T.proj(x, w, ws=ws), T.proj(xl, wl)
    old = ws.buf.numel()
    out, first = torch.empty_like(ref), torch.empty_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.proj(x, w, ws=ws, out=out)
    assert torch.equal(T.proj(xl, wl, ws=ws), large) and ws.buf.numel() > old
    others = [torch.full((old,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and all((o == 0xA5).all() for o in others)
        assert torch.equal(T.proj(xl, wl, ws=ws), large)
    # captured before the workspace has its size, and used before the first replay
    ws = T.Workspace("cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        T.proj(x, w, ws=ws, out=first)
        T.proj(x, w, ws=ws, out=out)
    assert torch.equal(T.proj(x, w, ws=ws), ref) and torch.equal(T.proj(xl, wl, ws=ws), large)
    for _ in range(3):
        first.zero_()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, ref) and torch.equal(out, ref)
    assert torch.equal(T.proj(x, w, ws=ws), ref) and ws.status()[0] == fnb.FN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 16])
def test_few_rows_whose_last_tiles_are_shared(M):
    """Few rows on the tile kernel with a k range long enough that the pairs
    share the last tile: the one case of a second kernel at so few rows."""
    K, N = 14336, 37900
    assert fnb.fn_workspace_size_proj(M, K, N) > 256
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.full((K, up8(N)), math.nan, dtype=torch.bfloat16, device="cuda")[:, :N]
    w.copy_(torch.randn(K, N, generator=g, device="cuda", dtype=torch.bfloat16) * K ** -0.5)
    r = torch.randn(M, N, generator=g, device="cuda")
    ws = T.Workspace("cuda")
    T.proj(x, w, residual=r, ws=ws)
    n = fnb.fn_kernel_launches()
    y = T.proj(x, w, residual=r, ws=ws)
    assert fnb.fn_kernel_launches() == n + 2
    n += 2
    for m, launches in ((1, 1), (16, 1), (17, 2)):             # the stream kernel
        T.proj(x[:1, :4096].expand(m, 4096).contiguous(), w[:4096, :4096], ws=ws)
        assert fnb.fn_kernel_launches() == n + launches
        n += launches
    torch.cuda.synchronize()
    for a in range(0, N, 4096):
        wd = w[:, a:a + 4096].double()
        ref = x.double() @ wd + r[:, a:a + 4096].double()
        tol = (8 + math.sqrt(K)) * 2 * U * (x.double().abs() @ wd.abs()) + 2 * U * ref.abs()
        assert ((y[:, a:a + 4096].double() - ref).abs() <= tol).all()
    assert ws.status()[0] == fnb.FN_OK and (ws.buf[:256] == 0).all()
