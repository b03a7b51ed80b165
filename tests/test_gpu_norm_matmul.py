"""GPU: gdn_rmsnorm_fp8 and gdn_fp8_matmul against their fp64 definitions (oracle/layer.py).

Tolerances.  E = 2^-24.  Norm: s is one fp32 addition; y three more roundings, the mean of D squares
(sqrt(D) E normwise, D/32 E at worst: the partial sums are short) and the root, so y is within
(16 + D / 32) E; the scale the same and one division.  q is y / scale rounded to e4m3: half a step is
2^-4 of the value, or 2^-10 where e4m3 is subnormal; the error of y / scale moves it by its own amount.
Matmul: products of e4m3 values are exact in fp32; sums of K terms and the scales: (K + 8) E of the
terms' magnitudes at worst, and half a step of the output's type."""
import pytest
import torch

import gated_delta_rule_71_b200 as gdn
import oracle
from oracle import layer
from tests._util import TOL_BF16, relerr

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
F8 = torch.float8_e4m3fn


def check_norm(x, w, r, q, sc, r_after, eps=1e-6):
    s, y, scales = (torch.from_numpy(t) for t in layer.rmsnorm(x, w, r, eps))
    D = x.shape[-1]
    tol = (16 + D / 32) * E
    if r is not None:
        half = torch.finfo(x.dtype).eps / 2
        assert ((r_after.cpu().double() - s).abs() <= (half * (1 + 2 * E) + E) * s.abs()).all()
    assert ((sc.cpu().double() - scales).abs() <= (tol + 2 * E) * scales).all()
    ex = scales.repeat_interleave(128, -1)[..., :D]
    t = y / ex
    err = (q.float().cpu().double() - t).abs()
    assert (err <= 2.0 ** -4 * t.abs().clamp(min=2.0 ** -6) + (2 * tol + 4 * E) * t.abs()).all()


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 127), (4, 128), (7, 129), (2, 1000), (9, 1001), (3, 2048),
                                    (2, 4104), (33, 4096), (2, 16384), (1, 16390), (1, 65536), (700, 256), (3001, 384), (1300, 4096),
                                    (1200, 8192), (1250, 2050)])
def test_norm(cuda_device, rows, D, res, ty):
    g = torch.Generator().manual_seed(D)
    x = torch.randn(rows, D, generator=g).to(ty).cuda()
    r = (3 * torch.randn(rows, D, generator=g)).to(ty).cuda() if res else None
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    r0 = r.clone() if res else None
    x0 = x.clone()
    q, sc = gdn.rmsnorm_fp8(x, w, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(x, x0)
    check_norm(x0, w, r0, q, sc, r)


def test_norm_of_strided_and_batched_rows(cuda_device):
    g = torch.Generator().manual_seed(1)
    w = torch.randn(264, generator=g).cuda()
    for off, width in ((0, 272), (8, 512), (3, 301)):
        base, rbase = (torch.randn(19, width, generator=g).bfloat16().cuda() for _ in range(2))
        x, r = base[:, off:off + 264], rbase[:, off:off + 264]
        keep, r0 = rbase.clone(), r.clone()
        q, sc = gdn.rmsnorm_fp8(x, w, residual=r, eps=1e-5)
        check_norm(x, w, r0, q, sc, r, eps=1e-5)
        assert torch.equal(rbase[:, :off], keep[:, :off]) and torch.equal(rbase[:, off + 264:], keep[:, off + 264:])
    x = torch.randn(2, 3, 5, 264, generator=g).cuda()
    q, sc = gdn.rmsnorm_fp8(x, w)
    assert q.shape == x.shape and sc.shape == (2, 3, 5, 3)
    check_norm(x, w, None, q, sc, None)


def test_norm_edges(cuda_device):
    x = torch.zeros(4, 300, device="cuda")
    w = torch.ones(300, device="cuda")
    x[1] = 1e18                       # its square is past fp32: no finite norm
    x[2, 5] = float("nan")
    x[3, :128] = 1.0                  # the other blocks of the row are zeros
    q, sc = gdn.rmsnorm_fp8(x, w)
    assert (sc[0] == 1).all() and not q[0].float().any()
    q1, s1 = gdn.rmsnorm_fp8(x[:1].contiguous(), w)
    assert torch.equal(q1.view(torch.uint8), q[:1].view(torch.uint8)) and torch.equal(s1, sc[:1])
    assert q[2].float().isnan().all() and sc[2].isnan().all()
    assert (q[3, :128].float() == 448).all() and not q[3, 128:].float().any() and (sc[3, 1:] == 1).all()
    # tiny values: eps carries the norm
    t = torch.full((1, 256), 1e-30, device="cuda")
    check_norm(t, w[:256].contiguous(), None, *gdn.rmsnorm_fp8(t, w[:256].contiguous()), None)
    e = gdn.rmsnorm_fp8(torch.empty(0, 300, device="cuda"), w)
    assert e[0].shape == (0, 300) and e[1].shape == (0, 3)


def test_norm_refusals(cuda_device):
    x, w = torch.zeros(2, 128, device="cuda"), torch.ones(128, device="cuda")
    for a, k in (((x.half(), w), {}), ((x, w[:64]), {}), ((x, w.bfloat16()), {}), ((x, w), dict(residual=x)),
                 ((x, w), dict(residual=x.bfloat16())), ((x, w), dict(residual=x[:1])), ((x, w), dict(eps=-1.0)),
                 ((x.expand(2, 2, 128), w), {}), ((x[:1].expand(5, 128), w), {}), ((x.t(), w), {}),
                 ((x, w), dict(scales=torch.empty(2, 2, device="cuda"))),
                 ((torch.zeros(1, 65544, device="cuda"), torch.ones(65544, device="cuda")), {})):
        with pytest.raises((ValueError, TypeError, gdn._lib.GdnError)):
            gdn.rmsnorm_fp8(*a, **k)


def operands(M, N, K, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    kb = -(-K // 128)
    q = lambda r: (100 * torch.randn(r, K + pad, generator=g)).clamp(-448, 448).to(F8).cuda()[:, :K]
    return (q(M), (0.01 * torch.exp(torch.randn(M, kb, generator=g))).cuda(), q(N),
            (0.01 * torch.exp(torch.randn(-(-N // 128), kb, generator=g))).cuda())


def check_matmul(ops, out):
    ref, mag = (torch.from_numpy(t) for t in layer.fp8_matmul(*ops))
    K = ops[0].shape[1]
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else E
    err = (out.cpu().double() - ref).abs()
    lim = half * ref.abs() + (K + 8) * E * mag
    assert (err <= lim).all(), float((err / lim).max())
    if out.dtype == torch.float32:  # normwise the roundings are independent
        assert err.norm() <= (8 + 2 * K ** 0.5) * E * mag.norm() / max(1.0, K ** 0.5)  + 4 * E * ref.norm()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 128, 128), (2, 130, 144), (16, 256, 512), (17, 1000, 2064),
                                   (33, 129, 272), (64, 512, 1024), (65, 384, 4096), (128, 136, 256), (129, 260, 384),
                                   (200, 640, 128), (257, 513, 640), (700, 1100, 400), (1, 4096, 2048),
                                   (300, 48, 8208), (5, 7, 13), (40, 300, 1001)])
def test_matmul(cuda_device, M, N, K, out):
    ops = operands(M, N, K, M + N + K)
    r = gdn.fp8_matmul(*ops, out_dtype=out)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check_matmul(ops, r)
    assert torch.equal(r, gdn.fp8_matmul(*ops, out_dtype=out))


def test_matmul_strides_batches_and_rows_left_alone(cuda_device):
    for pad in (16, 48, 5):
        ops = operands(70, 200, 256, pad, pad=pad)
        check_matmul(ops, gdn.fp8_matmul(*ops, out_dtype=torch.float32))
    a, sa, w, sw = operands(60, 200, 256, 3)
    buf = torch.full((62, 200), 9.0, dtype=torch.bfloat16, device="cuda")
    r = gdn.fp8_matmul(a.view(3, 20, 256), sa.view(3, 20, 2), w, sw, out=buf[1:61].view(3, 20, 200))
    check_matmul((a, sa, w, sw), r.view(60, 200))
    assert (buf[0] == 9).all() and (buf[61] == 9).all()
    assert gdn.fp8_matmul(a[:0], sa[:0], w, sw).shape == (0, 200)


def test_matmul_keeps_a_nan_in_its_row(cuda_device):
    a, sa, w, sw = operands(150, 260, 384, 4)
    ref = gdn.fp8_matmul(a, sa, w, sw)
    a.view(torch.uint8)[7, 3] = 0x7F
    sa[9, 1] = float("inf")
    r = gdn.fp8_matmul(a, sa, w, sw)
    keep = torch.ones(150, dtype=torch.bool)
    keep[[7, 9]] = False
    assert r[7].isnan().all() and not r[9].isfinite().any() and torch.equal(r[keep], ref[keep])


@pytest.mark.parametrize("M", [3, 300])
def test_matmul_streams_and_graph(cuda_device, M):
    one, two = operands(M, 520, 1024, 1), operands(M, 520, 1024, 2)
    want = [gdn.fp8_matmul(*o).clone() for o in (one, two)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for k, o in enumerate((one, two)):
            with torch.cuda.stream(streams[k]):
                got[k] = gdn.fp8_matmul(*o)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.fp8_matmul(*one)
    for src, w in ((two, want[1]),):
        for d, s in zip(one, src):
            d.copy_(s)
        graph.replay()
        assert torch.equal(out, w)
    del graph


def test_matmul_refusals(cuda_device):
    a, sa, w, sw = operands(4, 200, 256, 1)
    for bad in ((a.view(torch.uint8), sa, w, sw), (a, sa[:, :1], w, sw), (a, sa, w[:, :128], sw), (a, sa, w, sw[:1]),
                (a, sa.bfloat16(), w, sw), (a, sa, w.cpu(), sw), (a, sa, w.t(), sw), (a[:, ::2], sa, w, sw)):
        with pytest.raises((ValueError, TypeError, gdn._lib.GdnError)):
            gdn.fp8_matmul(*bad)
    with pytest.raises(TypeError):
        gdn.fp8_matmul(a, sa, w, sw, out_dtype=torch.float16)


def test_the_layer(cuda_device):
    """A state space layer end to end, as it is used: norm with the residual, projection, short convolution,
    scan with skip and gate, norm, projection; then a token of the same layer.  Against fp64 on the same 8-bit
    operands at each projection."""
    H, G, P, N, W, Dm, T = 4, 2, 64, 64, 4, 256, 150
    HP, GN = H * P, G * N
    C = HP + 2 * GN
    width = HP + C + 16  # [z | x B C | dt and padding to 16 bytes]
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g)
    q8 = lambda t: ((t / 0.01).clamp(-448, 448).to(F8).cuda(), torch.full((-(-t.shape[0] // 128), -(-t.shape[1] // 128)), 0.01).cuda())
    w_in, s_in = q8(r(width, Dm) / 4)
    w_out, s_out = q8(r(Dm, HP) / 4)
    nw1, nw2 = (1 + 0.1 * r(Dm)).cuda(), (1 + 0.1 * r(HP)).cuda()
    cw, cb = (r(C, W) / 2).cuda(), r(C).cuda()
    A_log, dtb, D = r(H).cuda(), (r(H) - 3).cuda(), r(H).cuda()
    x, res = r(T + 1, Dm).bfloat16().cuda(), r(T + 1, Dm).bfloat16().cuda()
    res0 = res.clone()

    q, s = gdn.rmsnorm_fp8(x, nw1, residual=res)
    check_norm(x, nw1, res0, q, s, res)
    row = gdn.fp8_matmul(q, s, w_in, s_in)
    check_matmul((q, s, w_in, s_in), row)
    z, xbc, dt = row[None, :, :HP], row[:, HP:HP + C], row[None, :, HP + C:HP + C + H]
    v, conv_state = gdn.conv1d_fwd(xbc[None, :T].contiguous(), cw, cb, activation=True, final_state=True)
    part = lambda a, b, k: v[..., a:b].unflatten(-1, (k, -1))
    args = dict(x=part(0, HP, H), dt=dt[:, :T], Bm=part(HP, HP + GN, G), Cm=part(HP + GN, C, G), A_log=A_log,
                dt_bias=dtb, D=D, z=z[:, :T].unflatten(-1, (H, P)))
    y, state = gdn.ssm_scan(**args)
    ry, rh, mag = (torch.from_numpy(t) for t in layer.ssm_scan(**args))
    u = 2.0 ** -8
    assert ((y.cpu().double() - ry).abs() <= u * ry.abs() + (u * (1 + u) + 2.0 ** -12) * mag).all()
    before = dict(conv_state=conv_state.clone(), state=state.clone())
    yt = gdn.ssm_decode_step(xbc[T:], dt[0, T:], cw, conv_state, A_log, dtb, state, H, G, P, N, D=D, z=z[0, T:],
                             conv_bias=cb)
    rt, rs, rc, ym, sm = (torch.from_numpy(t) for t in layer.ssm_decode_step(
        xbc[T:], dt[0, T:], cw, before["conv_state"], A_log, dtb, before["state"], H, G, P, N, D=D, z=z[0, T:],
        conv_bias=cb))
    assert ((yt.cpu().double() - rt).abs() <= u * rt.abs() + (96 + N) * E * ym).all()
    assert torch.equal(conv_state.cpu().double(), rc)
    assert ((state.cpu().double() - rs).abs() <= 64 * E * sm).all()
    both = torch.cat([y[0].flatten(1), yt.flatten(1)])
    q2, s2 = gdn.rmsnorm_fp8(both, nw2)
    out = gdn.fp8_matmul(q2, s2, w_out, s_out)
    check_norm(both, nw2, None, q2, s2, None)
    check_matmul((q2, s2, w_out, s_out), out)
    # the 8-bit path against the unquantised one: two roundings of 2^-4 / sqrt(3) in independent directions
    wf = (w_out.float() * 0.01).cpu().double()
    full = torch.from_numpy(layer.rmsnorm(both, nw2)[1]) @ wf.T
    assert (out.cpu().double() - full).norm() <= 2.0 ** -4 * full.norm()
    assert gdn.device_status() == 0


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1300, 1800, 400), (1281, 1805, 272), (2500, 1284, 128), (4097, 600, 1040),
                                   (300, 16001, 16)])
def test_matmul_of_prompts(cuda_device, M, N, K, out):
    # enough tiles of 128 tokens x 256 columns to fill the machine; ends inside a tile, rows of
    # the result on and off 16 bytes
    ops = operands(M, N, K, M + N + K)
    buf = torch.full((M + 2, N), 9.0, dtype=out, device="cuda")
    r = gdn.fp8_matmul(*ops, out_dtype=out, out=buf[1:M + 1])
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check_matmul(ops, r)
    assert (buf[0] == 9).all() and (buf[M + 1] == 9).all()
    assert torch.equal(r, gdn.fp8_matmul(*ops, out_dtype=out))


def test_norm_streams_and_graph(cuda_device):
    # the streamed form (many rows) and the register form on two streams at once, then replayed
    g = torch.Generator().manual_seed(6)
    sets = []
    for rows, D in ((2400, 1024), (40, 1024)):
        sets.append([torch.randn(rows, D, generator=g).bfloat16().cuda() for _ in range(2)] + [torch.ones(D, device="cuda")])
    want = [(r.clone(), *gdn.rmsnorm_fp8(x, w, residual=r)) for x, r, w in [(x, r.clone(), w) for x, r, w in sets]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [[r.clone() for _ in range(5)] for _, r, _ in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for i in range(5):
        for k, (x, _, w) in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                got[k] = gdn.rmsnorm_fp8(x, w, residual=res[k][i])
    torch.cuda.synchronize()
    for k in (0, 1):
        assert torch.equal(got[k][0].view(torch.uint8), want[k][1].view(torch.uint8)) and torch.equal(got[k][1], want[k][2])
    x, r, w = sets[0]
    live = r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, sc = gdn.rmsnorm_fp8(x, w, residual=live)
    for _ in range(2):
        live.copy_(r)
        graph.replay()
        assert torch.equal(q.view(torch.uint8), want[0][1].view(torch.uint8)) and torch.equal(sc, want[0][2])
    del graph


def test_offsets_behind_two_to_the_31(cuda_device):
    D, rows = 8192, 262400  # 2^31 elements and more: the last rows are what they are by themselves
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    w = torch.ones(D, device="cuda")
    r = torch.zeros_like(x)
    q, sc = gdn.rmsnorm_fp8(x, w, residual=r)
    q1, sc1 = gdn.rmsnorm_fp8(x[-1300:], w, residual=torch.zeros_like(x[-1300:]))
    assert torch.equal(q[-1300:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(sc[-1300:], sc1)
    assert torch.equal(r[-1300:], x[-1300:])
    del x, r, q
    a, sa, w, sw = operands(65600, 32776, 16, 8)
    out = gdn.fp8_matmul(a, sa, w, sw)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check_matmul((a[-40:], sa[-40:], w, sw), out[-40:])


@pytest.mark.parametrize("rows,D", [(1, 300), (1, 296), (1300, 256), (1300, 1024)])
def test_norm_of_values_whose_scale_underflows(cuda_device, rows, D):
    # y near 2^-143: max|y| / 448 is 0 in fp32, so the scale is 1 and the values round to 0
    x = torch.ones(rows, D, device="cuda")
    x[:, 1::2] = 0.0
    q, sc = gdn.rmsnorm_fp8(x, torch.full((D,), 1e-43, device="cuda"))
    assert (sc == 1).all() and not q.float().any()
    # at 448 units of the smallest fp32 number the scale is that number, and the values are exact
    w = torch.full((D,), 448 * 2.0 ** -149, device="cuda")
    x[:] = 1.0
    q, sc = gdn.rmsnorm_fp8(x, w, eps=0.0)
    assert (sc == 2.0 ** -149).all() and (q.float() == 448).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(20000, 384), (40001, 256), (75777, 400)])
@pytest.mark.parametrize("M", [1, 17, 64, 100])
def test_matmul_of_few_tokens_onto_a_wide_result(cuda_device, M, N, K, out):
    # more tiles of 128 weight rows than SMs, and more than CTAs that fit: one CTA walks several, over odd
    # and even numbers of K blocks
    ops = operands(M, N, K, M + N + K)
    buf = torch.full((M + 2, N), 9.0, dtype=out, device="cuda")
    r = gdn.fp8_matmul(*ops, out_dtype=out, out=buf[1:M + 1])
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check_matmul(ops, r)
    assert (buf[0] == 9).all() and (buf[M + 1] == 9).all()
    assert torch.equal(r, gdn.fp8_matmul(*ops, out_dtype=out))


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("rows,D", [(1300, 256), (5000, 64), (2001, 8), (1185, 264), (1300, 512), (1300, 1000), (1300, 2048),
                                    (1300, 4264)])
def test_norm_of_many_rows(cuda_device, rows, D, res, ty):
    # the forms of many rows, one warp a row and streamed, each width of them: contiguous rows, and rows of a wider tensor
    g = torch.Generator().manual_seed(D)
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    for width, off in ((D, 0), (D + 24, 8)):
        base = torch.randn(rows, width, generator=g).to(ty).cuda()
        rbase = (3 * torch.randn(rows, width, generator=g)).to(ty).cuda() if res else None
        x, keep = base[:, off:off + D], base.clone()
        r = rbase[:, off:off + D] if res else None
        r0, rkeep = (r.clone(), rbase.clone()) if res else (None, None)
        q, sc = gdn.rmsnorm_fp8(x, w, residual=r)
        torch.cuda.synchronize()
        assert gdn.device_status() == 0 and torch.equal(base, keep)
        check_norm(x, w, r0, q, sc, r)
        if res:
            rkeep[:, off:off + D] = rbase[:, off:off + D]
            assert torch.equal(rbase, rkeep)


def test_norm_of_rows_past_fp32(cuda_device):
    # a row whose sum of squares is past fp32 has no finite norm in it: zeros, under scales of one
    x = torch.ones(1300, 256, device="cuda")
    x[[1, 77]] = 1e20
    w = torch.ones(256, device="cuda")
    for rows in (3, 1300):
        q, sc = gdn.rmsnorm_fp8(x[:rows], w)
        for r in (1, 77):
            if r < rows:
                assert not q[r].float().any() and (sc[r] == 1).all()
        assert (q[[0, 2]].float() == 448).all()


def test_norm_residuals_of_two_streams(cuda_device):
    g = torch.Generator().manual_seed(16)
    sets = [[torch.randn(rows, D, generator=g).bfloat16().cuda() for _ in range(2)] for rows, D in ((2400, 1024), (3000, 256), (40, 1024))]
    want = [(x.float() + r.float()).bfloat16() for x, r in sets]
    live = [[r.clone() for _ in range(5)] for _, r in sets]
    ones = torch.ones(1024, device="cuda")
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for i in range(5):
        for k, (x, _) in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                gdn.rmsnorm_fp8(x, ones[:x.shape[1]], residual=live[k][i])
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[k]) for k in range(len(sets)) for t in live[k])


def test_projection_into_the_product_rule(cuda_device):
    """Norm and projection in front of the library's other recurrence: a prompt through gdp_prefill, then a
    token through gdp_decode_layer_step, both on slices of the projected rows."""
    M, H, G, P, N, W, Dm, T = 2, 4, 2, 128, 128, 4, 256, 97
    vals, C = M * H * P, M * H * P + M * G * N + G * N
    width = C + 16  # [values | keys | queries | ba and padding to 16 bytes]
    g = torch.Generator().manual_seed(15)
    r = lambda *s: torch.randn(s, generator=g)
    w = (100 * r(width, Dm)).clamp(-448, 448).to(F8).cuda()
    ws = torch.full((-(-width // 128), 2), 0.01 / 16)
    ws[vals // 128:C // 128] /= N ** 0.5  # keys and queries of about unit norm
    ws = ws.cuda()
    x, res = r(T + 3, Dm).bfloat16().cuda(), r(T + 3, Dm).bfloat16().cuda()
    A_log, dtb = (torch.rand(H, generator=g) * 2).cuda(), (r(H) - 3).cuda()
    q, s = gdn.rmsnorm_fp8(x, (1 + 0.1 * r(Dm)).cuda(), residual=res)
    row = gdn.fp8_matmul(q, s, w, ws)
    check_matmul((q, s, w, ws), row)
    xs, ba = row[:, :C], row[:, C:C + M * H + H]
    o, hT = gdn.gdp_prefill(xs[None, :T], ba[None, :T], A_log, dtb, M, H, G, P, N)
    c = lambda t: t.cpu()
    ro, rh = oracle.gdp_prefill(c(xs[None, :T]), c(ba[None, :T]), c(A_log), c(dtb), M, H, G, P, N)
    assert relerr(o, ro) <= TOL_BF16 and relerr(hT, rh) <= TOL_BF16
    # three requests' tokens, each on a copy of that state
    st = hT.expand(3, -1, -1, -1).contiguous()
    cw, cb, cs = (r(C, W) / 2).cuda(), r(C).cuda(), r(3, C, W - 1).bfloat16().cuda()
    y, rcs = oracle.conv1d_update(c(xs[T:]), c(cw), c(cs), bias=c(cb), activation=True)
    ro, rs = oracle.gdp_decode_step_indexed(torch.from_numpy(y).float().bfloat16().reshape(3, 1, C), c(ba[T:]).reshape(3, 1, -1),
                                            c(A_log), c(dtb), c(st), torch.arange(3, dtype=torch.int32), M, H, G, P, N)
    out = gdn.gdp_decode_layer_step(xs[T:], ba[T:], cw, cs, A_log, dtb, st, M, H, G, P, N, conv_bias=cb)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    assert relerr(out, ro) <= TOL_BF16 and relerr(st, rs) <= TOL_BF16
    assert torch.equal(cs.cpu().float(), torch.from_numpy(rcs).float())


def test_norm_of_rows_that_vanish_in_fp32(cuda_device):
    # with eps = 0 a row whose squares are 0 in fp32 has no finite scale; the smallest eps gives it one
    x = torch.ones(3, 256, device="cuda")
    x[1] = 1e-30
    w = torch.ones(256, device="cuda")
    q, sc = gdn.rmsnorm_fp8(x, w, eps=0.0)
    assert not sc[1].isfinite().any() and (sc[[0, 2]] == sc[0, 0]).all() and (q[[0, 2]].float() == 448).all()
    check_norm(x, w, None, *gdn.rmsnorm_fp8(x, w, eps=1e-30), None, eps=1e-30)
