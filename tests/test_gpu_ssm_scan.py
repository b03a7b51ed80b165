"""GPU: gdn_ssm_scan against its fp64 definition (oracle/layer.py), token by token.

Tolerances.  u = 2^-8 is half a step of bf16 and e = 2^-24 half a step of fp32, both relative.
* bf16 y: the pair weights of a chunk, the state that multiplies C, and y itself are each rounded to
  bf16 once.  A term of y goes through one of the first two, so |dy| <= u |y| + u (1 + u) mag, mag
  being the sum of the magnitudes of y's terms; 2^-12 mag more covers the fp32 arithmetic (decays as
  differences of sums up to 2^9 in 32 bits: 2^9 e relative to a term, twice).  Normwise the three
  roundings are independent and uniform, so their squares add: at most sqrt(2) of one rounding's rms
  (u / sqrt(3)) for each part, below u in all.
* fp32 y, and every state: products of fp32 factors, each of a handful of operations (32 e covers
  softplus, exp, their arguments and the products), and one rounding (and one decay) a token that a
  term passes.  Worst case 3 T e; normwise the roundings are independent: 2 sqrt(T) e.
"""
import math

import pytest
import torch

import gated_delta_rule_71_b200 as gdn
from oracle import layer

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24


def make(B, T, H, G, P, N, ty, seed, lens=None, D=True, z=True, h0=True, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    row = torch.nn.functional.silu(r(B, T, H * P + 2 * G * N)).to(ty).to(dev)
    n_seq = len(lens) if lens is not None else B
    d = dict(x=row[..., :H * P].unflatten(-1, (H, P)), Bm=row[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
             Cm=row[..., H * P + G * N:].unflatten(-1, (G, N)), dt=r(B, T, H).to(ty).to(dev),
             A_log=(torch.rand(H, generator=g) * math.log(16.0)).to(dev),
             dt_bias=torch.log(torch.expm1(torch.exp(torch.rand(H, generator=g) * math.log(100.0) - math.log(1e3)))).to(dev),
             D=r(H).to(dev) if D else None, z=r(B, T, H, P).to(ty).to(dev) if z else None,
             h0=0.1 * r(n_seq, H, N, P).to(dev) if h0 else None,
             cu_seqlens=None if lens is None else torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(),
                                                               dtype=torch.int32, device=dev))
    return d


def check(d, y, hT):
    ry, rh, mag = (torch.from_numpy(t) for t in layer.ssm_scan(**d))
    T = d["x"].shape[1]
    err = (y.cpu().double() - ry).abs()
    if d["x"].dtype == torch.bfloat16:
        lim = U * ry.abs() + (U * (1 + U) + 2.0 ** -12) * mag + 1e-30
        assert (err <= lim).all(), f"y: {float((err / lim).max()):.3g} of the bound"
        assert err.norm() <= U * ry.norm()
    else:
        lim = (32 + 3 * T) * E * mag + 1e-30
        assert (err <= lim).all(), f"y: {float((err / lim).max()):.3g} of the bound"
        assert err.norm() <= (32 + 2 * math.sqrt(T)) * E * mag.norm()
    if hT is not None:
        eh = (hT.cpu().double() - rh)
        assert eh.norm() <= (32 + 2 * math.sqrt(T)) * E * rh.norm() + 1e-30, float(eh.norm() / rh.norm())


CASES = [  # B, T, H, G, P, N, lens
    (1, 1, 2, 1, 64, 128, None), (2, 2, 2, 2, 64, 64, None), (1, 127, 4, 2, 64, 128, None),
    (1, 128, 3, 1, 64, 128, None), (2, 129, 4, 1, 128, 128, None), (1, 300, 2, 1, 32, 32, None),
    (3, 130, 6, 2, 32, 64, None), (1, 257, 2, 2, 128, 64, None), (1, 200, 4, 1, 64, 32, None),
    (1, 260, 5, 5, 64, 128, None), (1, 515, 3, 1, 128, 32, [0, 1, 127, 128, 129, 0, 130, 0]),
    (1, 700, 4, 2, 64, 64, [5, 600, 0, 95]), (1, 3, 4, 2, 64, 128, [1, 1, 1])]


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,H,G,P,N,lens", CASES)
def test_matches_the_definition(cuda_device, B, T, H, G, P, N, lens, ty):
    d = make(B, T, H, G, P, N, ty, 100 + T, lens)
    y, hT = gdn.ssm_scan(**d)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check(d, y, hT)


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,z,h0", [(False, False, False), (True, False, False), (False, True, True)])
def test_without_the_options(cuda_device, D, z, h0, ty):
    d = make(2, 150, 4, 2, 64, 128, ty, 7, D=D, z=z, h0=h0)
    y, hT = gdn.ssm_scan(**d)
    check(d, y, hT)
    y2, none = gdn.ssm_scan(**d, output_final_state=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("lens", [None, [700, 1500, 0, 33, 2367]])
def test_long_sequences_split_over_their_length(cuda_device, lens):
    # few heads: the sequence itself has to fill the machine
    d = make(1, 4600, 2, 1, 64, 64, torch.bfloat16, 21, lens)
    d["A_log"] -= 3.0  # slow decay: what a split loses would show for long
    y, hT = gdn.ssm_scan(**d)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check(d, y, hT)
    for _ in range(3):
        y2, hT2 = gdn.ssm_scan(**d)
        assert torch.equal(y, y2) and torch.equal(hT, hT2)


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
def test_empty_batch_and_zero_length(cuda_device, ty):
    d = make(2, 0, 2, 1, 64, 64, ty, 3)
    y, hT = gdn.ssm_scan(**d)
    assert y.shape == (2, 0, 2, 64) and torch.equal(hT, d["h0"])
    d = make(1, 0, 2, 1, 64, 64, ty, 3, lens=[0, 0, 0])
    assert torch.equal(gdn.ssm_scan(**d)[1], d["h0"])
    d["h0"] = None
    assert not gdn.ssm_scan(**d)[1].any()


def test_continuation(cuda_device):
    d = make(1, 333, 4, 2, 64, 128, torch.bfloat16, 5)
    y, hT = gdn.ssm_scan(**d)
    cut = lambda a, b: {k: (v[:, a:b] if k in ("x", "Bm", "Cm", "dt", "z") else v) for k, v in d.items()}
    y1, h1 = gdn.ssm_scan(**cut(0, 200))
    y2, h2 = gdn.ssm_scan(**{**cut(200, 333), "h0": h1})
    assert (hT - h2).norm() <= 80 * E * hT.norm()
    ry, _, mag = (torch.from_numpy(t) for t in layer.ssm_scan(**d))
    err = (torch.cat([y1, y2], 1).cpu().double() - ry).abs()
    assert (err <= U * ry.abs() + (U * (1 + U) + 2.0 ** -12) * mag).all()


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64), (32, 32)])
def test_rows_of_any_alignment(cuda_device, P, N):
    # the same values in rows that start on any 2-byte address give the same result to tolerance
    d = make(2, 140, 2, 1, P, N, torch.bfloat16, 9)
    w = 2 * P + 2 * N
    wide = torch.zeros(2, 140, w + 5, dtype=torch.bfloat16, device="cuda")
    wide[..., 3:3 + 2 * P] = d["x"].flatten(2)
    wide[..., 3 + 2 * P:3 + 2 * P + N] = d["Bm"].flatten(2)
    wide[..., 3 + 2 * P + N:3 + w] = d["Cm"].flatten(2)
    e = dict(d, x=wide[..., 3:3 + 2 * P].unflatten(-1, (2, P)), Bm=wide[..., 3 + 2 * P:3 + 2 * P + N].unflatten(-1, (1, N)),
             Cm=wide[..., 3 + 2 * P + N:3 + w].unflatten(-1, (1, N)))
    y, hT = gdn.ssm_scan(**e)
    check(e, y, hT)


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_poisoned_sequence_reaches_no_other(cuda_device, ty, bad):
    lens = [70, 130, 1, 200]
    d = make(1, 401, 2, 1, 64, 128, ty, 13, lens)
    ref = [t.clone() for t in gdn.ssm_scan(**d)]
    for key in ("x", "Bm", "Cm", "dt", "z"):
        d[key] = d[key].clone()
        d[key][:, 70:200] = bad
    d["h0"][1] = bad
    y, hT = gdn.ssm_scan(**d)
    keep = torch.ones(401, dtype=torch.bool)
    keep[70:200] = False
    assert torch.equal(y[:, keep], ref[0][:, keep])
    assert torch.equal(hT[[0, 2, 3]], ref[1][[0, 2, 3]])
    assert y[:, 70:200].isnan().any() or y[:, 70:200].isinf().any()


def test_extreme_decays(cuda_device):
    # steps that forget everything and steps that forget nothing
    d = make(1, 400, 4, 1, 64, 64, torch.bfloat16, 17)
    d["dt"] = d["dt"].clone()
    d["dt"][:, 100:140] = 60.0
    d["dt"][:, 200:390] = -80.0
    d["A_log"] = torch.tensor([3.0, -20.0, 0.0, 2.7], device="cuda")
    y, hT = gdn.ssm_scan(**d)
    assert y.isfinite().all()
    check(d, y, hT)


def test_rows_behind_the_last_sequence_stay(cuda_device):
    d = make(1, 300, 2, 1, 64, 64, torch.bfloat16, 19, lens=[100, 100])
    out = torch.full((1, 300, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    gdn.ssm_scan(**d, out=out)
    assert (out[:, 200:] == 7.0).all() and not (out[:, :200] == 7.0).all()


def test_streams_graph_and_replay(cuda_device):
    a, b = (make(1, 900, 2, 1, 64, 64, torch.bfloat16, s, lens=[300, 600]) for s in (31, 32))
    want = [[t.clone() for t in gdn.ssm_scan(**d)] for d in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(5):
        for k, (s, d) in enumerate(((s1, a), (s2, b))):
            with torch.cuda.stream(s):
                got[k] = gdn.ssm_scan(**d)
    torch.cuda.synchronize()
    for k in (0, 1):
        assert torch.equal(got[k][0], want[k][0]) and torch.equal(got[k][1], want[k][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.ssm_scan(**a)
    for k, d in ((1, b), (0, a)):
        src = {key: v.clone() for key, v in d.items() if isinstance(v, torch.Tensor)} if k else None
        keep = {key: v.clone() for key, v in a.items() if isinstance(v, torch.Tensor)} if k else keep
        for key, v in (src or keep).items():
            a[key].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[k][0]) and torch.equal(out[1], want[k][1])
    del graph


def test_refusals(cuda_device):
    d = make(1, 8, 2, 1, 64, 64, torch.bfloat16, 1)
    for change in (dict(dt=d["dt"].float()), dict(Bm=d["Bm"][:, :7]), dict(D=d["D"][:1]), dict(z=d["z"][..., :32]),
                   dict(h0=d["h0"][:, :1]), dict(x=d["x"].transpose(-1, -2)), dict(A_log=d["A_log"].cpu()),
                   dict(x=d["x"].half(), dt=d["dt"].half(), Bm=d["Bm"].half(), Cm=d["Cm"].half(), z=None),
                   dict(out=d["x"]), dict(workspace=torch.empty(8))):
        with pytest.raises((ValueError, TypeError, gdn._lib.GdnError)):
            gdn.ssm_scan(**{**d, **change})
    x = d["x"].expand(2, 8, 2, 64)
    with pytest.raises(ValueError):  # rows of the two sequences are the same memory
        gdn.ssm_scan(x, *(d[k].expand(2, *d[k].shape[1:]) for k in ("dt", "Bm", "Cm")), d["A_log"], d["dt_bias"])


@pytest.mark.parametrize("lens", [[(7 * i * i) % 10 for i in range(700)], [(5 * i) % 4 for i in range(300)] + [4000]])
def test_many_short_sequences(cuda_device, lens):
    d = make(1, sum(lens), 2, 1, 64, 64, torch.bfloat16, 41, lens)
    y, hT = gdn.ssm_scan(**d)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check(d, y, hT)


def test_rows_behind_two_to_the_31(cuda_device):
    # y and x pass 2^31 elements; the last sequence is what it is by itself
    T, H, P = 524416, 32, 128
    d = make(1, 300, H, 1, P, 64, torch.bfloat16, 43, lens=[300], h0=False)
    g = torch.Generator("cuda").manual_seed(1)
    big = {}
    for k in ("x", "Bm", "Cm", "dt", "z"):
        t = torch.empty((1, T, *d[k].shape[2:]), dtype=torch.bfloat16, device="cuda")
        if k == "z":
            t.fill_(1.0)
        else:
            t.normal_(generator=g)
        t[:, T - 300:] = d[k]
        big[k] = t
    y, hT = gdn.ssm_scan(**{**d, **big, "cu_seqlens": torch.tensor([0, T - 300, T], dtype=torch.int32, device="cuda")})
    y1, h1 = gdn.ssm_scan(**d)
    assert gdn.device_status() == 0
    assert torch.equal(y[:, T - 300:], y1) and torch.equal(hT[1:], h1)
    check(d, y1, h1)


@pytest.mark.parametrize("lens", [[1] * 14 + [100], [8] * 13, [0, 3, 2, 5, 1, 4, 3, 0, 6, 2, 5, 1, 4]])
def test_a_prompt_packed_with_short_sequences(cuda_device, lens):
    # a prompt's result does not depend on what it is packed with, and it is not walked token by token
    T = sum(lens)
    d = make(1, T, 16, 2, 64, 64, torch.bfloat16, 47, lens)
    y, hT = gdn.ssm_scan(**d)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check(d, y, hT)
    n = lens[-1]
    if n > 32:
        alone = {k: v[:, T - n:] if k in ("x", "Bm", "Cm", "dt", "z") else v for k, v in d.items()}
        y1, h1 = gdn.ssm_scan(**{**alone, "h0": d["h0"][-1:], "cu_seqlens": None})
        assert torch.equal(y[:, T - n:], y1) and torch.equal(hT[-1:], h1)


@pytest.mark.parametrize("B,T,lens", [(2, 1600, None), (1, 2601, [700, 1, 1500, 0, 400])])
@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("H,G,P,N", [(6, 2, 64, 128), (4, 2, 128, 128), (3, 1, 128, 64), (10, 2, 32, 32)])
def test_cut_sequences_of_every_form(cuda_device, H, G, P, N, h0, B, T, lens):
    # the segments' sums, their chain and the walk from them: one head or two a unit, an odd number of heads
    # a group (a unit with a missing head), several units, and each width of the state
    assert gdn.ssm_scan_workspace_size(len(lens or []) or B, B * T, H, G, P, N) > 0
    d = make(B, T, H, G, P, N, torch.bfloat16, 51, lens, h0=h0)
    d["A_log"] -= 3.0  # slow decay: what a cut loses would show for long
    y, hT = gdn.ssm_scan(**d)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check(d, y, hT)
    y2, hT2 = gdn.ssm_scan(**d)
    assert torch.equal(y, y2) and torch.equal(hT, hT2)


@pytest.mark.parametrize("B,T,H,G,P,N,cut,lens", [
    (37, 8192, 8, 4, 64, 64, False, None), (74, 8192, 2, 2, 128, 128, False, None), (1, 131072, 32, 1, 64, 64, True, None),
    (2, 40000, 4, 1, 64, 128, True, None), (1, 16384, 296, 148, 64, 64, False, [300, 8000, 0, 5000, 3084])])
def test_states_that_do_not_decay(cuda_device, B, T, H, G, P, N, cut, lens):
    # The final state of a head whose decay is nothing, or slow, is a sum over the whole sequence: to fp32's
    # bound, in sequences that one CTA walks and in cut ones.  hT = sum_t e^(sum of g behind t) dt_t B_t x_t^T.
    g = torch.Generator("cuda").manual_seed(61)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    row = torch.nn.functional.silu(r(B, T, H * P + 2 * G * N)).bfloat16()
    n_seq = B if lens is None else len(lens)
    if cut:
        assert gdn.ssm_scan_workspace_size(B, B * T, H, G, P, N) > 0
    A_log = torch.full((H,), -20.0, device="cuda")
    A_log[1::2] = -4.0
    d = dict(x=row[..., :H * P].unflatten(-1, (H, P)), Bm=row[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
             Cm=row[..., H * P + G * N:].unflatten(-1, (G, N)), dt=r(B, T, H).bfloat16(), A_log=A_log,
             dt_bias=torch.full((H,), -4.0, device="cuda"), h0=0.1 * r(n_seq, H, N, P))
    if lens is not None:
        d["cu_seqlens"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    hT = gdn.ssm_scan(**d)[1]
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    ends = [(b * T, (b + 1) * T) for b in range(B)] if lens is None else list(zip(d["cu_seqlens"].tolist(), d["cu_seqlens"].tolist()[1:]))
    x, Bm, dt = d["x"].flatten(0, 1), d["Bm"].flatten(0, 1), d["dt"].flatten(0, 1)
    for s in sorted({0, 1 % n_seq, n_seq // 2, n_seq - 1}):
        for h in (0, 1, H - 1):
            a, b = ends[s]
            step = torch.nn.functional.softplus(dt[a:b, h].double() + d["dt_bias"][h].double())
            decay = -torch.exp(A_log[h].double()) * step
            behind = decay.flip(0).cumsum(0).flip(0)
            w = torch.exp(behind - decay) * step
            ref = Bm[a:b, h // (H // G)].double().T @ (w[:, None] * x[a:b, h].double())
            ref += d["h0"][s, h].double() * (torch.exp(behind[0]) if b > a else 1.0)
            err = (hT[s, h].double() - ref).norm()
            assert err <= (32 + 2 * math.sqrt(b - a)) * E * ref.norm(), (s, h, float(err / ref.norm() / E))


@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("P,N", [(64, 128), (128, 64), (64, 64)])
def test_what_stands_behind_a_prompt_in_a_padded_batch(cuda_device, P, N, bad, ty):
    # dt, Bm, Cm and z of the tokens behind the prompts hold garbage, and x from the next block of 128 on (bf16):
    # the prompts' y is what it is without them
    d = make(3, 430, 4, 2, P, N, ty, 73)
    ends = (150, 257, 384)
    for key in ("x", "Bm", "Cm", "dt", "z"):
        d[key] = d[key].clone()
        for b, n in enumerate(ends):
            d[key][b, -(-n // 128) * 128 if key == "x" and ty == torch.bfloat16 else n:] = bad
    y, _ = gdn.ssm_scan(**d)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    for b, n in enumerate(ends):
        one = {k: v[b:b + 1, :n] if k in ("x", "Bm", "Cm", "dt", "z") else v for k, v in d.items()}
        one["h0"] = d["h0"][b:b + 1]
        check(one, y[b:b + 1, :n], None)
