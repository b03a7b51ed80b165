"""GPU: gdn_ssm_decode_step against its fp64 definition (oracle/layer.py).

Tolerances: the step is fp32 throughout and rounded to bf16 once, at y.  E = 2^-24.  A convolved channel
is a sum of at most 4 taps and a bias, which may cancel: its error is relative to the sum of their
magnitudes (5 roundings, then SiLU, whose slope is below 1.1, within 8 E: 16 E).  A state element adds
the products of two such with dt (softplus, 16 E) to a decayed state (exp and its argument, 16 E), a few
roundings each: 64 E of the magnitudes.  y sums N of them times a third channel: (96 + N) E of the
magnitudes, the gate included, and half a bf16 step, 2^-8 |y|.  The conv window is moved bit for bit."""
import pytest
import torch

import gated_delta_rule_71_b200 as gdn
from oracle import layer

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def make(n, slots, H, G, P, N, W=4, seed=0, z=True, D=True, bias=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    C = H * P + 2 * G * N
    row = r(n, H * P + C + H + wide).bfloat16().cuda()  # the projected row [z | x B C | dt | ...]
    d = dict(row=row[:, H * P:H * P + C], dt=row[:, H * P + C:H * P + C + H], conv_w=(r(C, W) / W ** 0.5).cuda(),
             conv_state=r(slots, C, W - 1).bfloat16().cuda(), A_log=r(H).cuda(), dt_bias=(r(H) - 3).cuda(),
             state=(0.1 * r(slots, H, N, P)).cuda(), H=H, G=G, P=P, N=N, D=r(H).cuda() if D else None,
             z=row[:, :H * P] if z else None, conv_bias=r(C).cuda() if bias else None)
    return d


def clone(d):
    return {k: v.clone() if k in ("state", "conv_state") else v for k, v in d.items()}


def check(d, before):
    ry, rs, rc, ym, sm = (torch.from_numpy(t) for t in layer.ssm_decode_step(**before))
    y, st, cs = d["y"].cpu().double(), d["state"].cpu().double(), d["conv_state"].cpu().double()
    assert torch.equal(cs, rc)
    over = lambda err, lim: float((err / (lim + 1e-30)).max())
    assert over((st - rs).abs(), 64 * E * sm) <= 1
    assert over((y - ry).abs(), 2.0 ** -8 * ry.abs() + (96 + before["N"]) * E * ym) <= 1


@pytest.mark.parametrize("n,H,G,P,N,W", [(1, 2, 1, 64, 128, 4), (5, 4, 2, 128, 128, 4), (9, 3, 1, 32, 32, 2),
                                         (17, 8, 8, 64, 64, 3), (3, 6, 2, 128, 32, 4), (2, 1, 1, 32, 128, 1),
                                         (33, 2, 1, 64, 32, 4), (4, 5, 5, 128, 64, 4)])
def test_matches_the_definition(cuda_device, n, H, G, P, N, W):
    d = make(n, n + 3, H, G, P, N, W, seed=n)
    d["state_indices"] = torch.randperm(n + 3, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32).cuda()
    before = clone(d)
    d["y"] = gdn.ssm_decode_step(**d)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    check(d, before)


@pytest.mark.parametrize("z,D,bias,wide", [(False, False, False, 0), (True, False, True, 1), (False, True, False, 3)])
def test_options_and_odd_strides(cuda_device, z, D, bias, wide):
    d = make(6, 6, 4, 2, 64, 64, seed=2, z=z, D=D, bias=bias, wide=wide)
    before = clone(d)
    d["y"] = gdn.ssm_decode_step(**d)
    check(d, before)
    d2 = clone(before)
    y2 = gdn.ssm_decode_step(**d2, activation=True)
    assert torch.equal(y2, d["y"]) and torch.equal(d2["state"], d["state"])


def test_no_activation(cuda_device):
    d = make(4, 4, 2, 1, 64, 64, seed=8)
    before = clone(d)
    y = gdn.ssm_decode_step(**d, activation=False)
    ry, rs, _, ym, sm = (torch.from_numpy(t) for t in layer.ssm_decode_step(**before, activation=False))
    assert ((y.cpu().double() - ry).abs() <= 2.0 ** -8 * ry.abs() + (96 + 64) * E * ym).all()
    assert ((d["state"].cpu().double() - rs).abs() <= 64 * E * sm).all()


def test_padding_and_slots_out_of_range(cuda_device):
    d = make(8, 20, 4, 2, 64, 128, seed=4)
    idx = torch.tensor([3, -1, 7, 20, 0, -5, 19, 11], dtype=torch.int32)
    d["state_indices"] = idx.cuda()
    before = clone(d)
    d["y"] = gdn.ssm_decode_step(**d)
    assert gdn.device_status() == 1 and gdn.device_status() == 0
    assert not d["y"][[1, 3, 5]].any()
    used = [3, 7, 0, 19, 11]
    rest = [s for s in range(20) if s not in used]
    assert torch.equal(d["state"][rest], before["state"][rest])
    assert torch.equal(d["conv_state"][rest], before["conv_state"][rest])
    before["state_indices"] = torch.where(idx >= 20, -1, idx).cuda()
    check(d, before)


def test_tokens_in_a_row_and_in_a_graph(cuda_device):
    # the same tokens, called one by one and replayed from one graph with one workspace
    d = make(3, 5, 4, 1, 64, 64, seed=6)
    d["state_indices"] = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    ws = torch.empty(gdn.ssm_decode_step_workspace_size(3, 4, 1, 64, 64), dtype=torch.uint8, device="cuda")
    a, b = clone(d), clone(d)
    gen = torch.Generator().manual_seed(9)
    base = d["row"]._base if d["row"]._base is not None else d["row"]
    tokens = [torch.randn(base.shape, generator=gen).bfloat16().cuda() for _ in range(4)]
    ref = []
    for t in tokens:
        base.copy_(t)
        before = clone(a)
        a["y"] = gdn.ssm_decode_step(**{k: v for k, v in a.items() if k != "y"})
        check(a, {k: v for k, v in before.items() if k != "y"})
        ref.append(a["y"].clone())
    warm = clone(d)
    gdn.ssm_decode_step(**warm, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gdn.ssm_decode_step(**b, workspace=ws)
    for t, r in zip(tokens, ref):
        base.copy_(t)
        graph.replay()
        assert torch.equal(y, r)
    assert torch.equal(a["state"], b["state"]) and torch.equal(a["conv_state"], b["conv_state"])
    del graph


def test_one_more_token_of_the_scan(cuda_device):
    # prompt through conv1d_fwd and ssm_scan, then one token, against the scan of all of them
    H, G, P, N, W, T = 4, 2, 64, 64, 4, 130
    C = H * P + 2 * G * N
    g = torch.Generator().manual_seed(12)
    row = torch.randn(1, T, C, generator=g).bfloat16().cuda()
    dt = torch.randn(1, T, H, generator=g).bfloat16().cuda()
    w, bias = (torch.randn(C, W, generator=g) / 2).cuda(), torch.randn(C, generator=g).cuda()
    A_log, dtb = torch.randn(H, generator=g).cuda(), (torch.randn(H, generator=g) - 3).cuda()

    def scan(T):
        v, fin = gdn.conv1d_fwd(row[:, :T].contiguous(), w, bias, activation=True, final_state=True)
        s = lambda a, b, k: v[..., a:b].unflatten(-1, (k, -1))
        y, hT = gdn.ssm_scan(s(0, H * P, H), dt[:, :T], s(H * P, H * P + G * N, G), s(H * P + G * N, C, G), A_log, dtb)
        return y, hT, fin
    y, hT, fin = scan(T)
    _, h, cs = scan(T - 1)
    yt = gdn.ssm_decode_step(row[:, -1], dt[:, -1], w, cs, A_log, dtb, h, H, G, P, N, conv_bias=bias)
    # the scan's last token went through a bf16 convolution: x, B and C off by 2^-8 each
    assert (yt - y[:, -1]).float().norm() <= 4 * 2.0 ** -8 * y[:, -1].float().norm()
    assert (h - hT).norm() <= 2 * 2.0 ** -8 * hT.norm()
    assert torch.equal(cs, fin)


def test_refusals(cuda_device):
    d = make(4, 4, 2, 1, 64, 64, seed=1)
    for change in (dict(row=d["row"][:, :-1]), dict(dt=d["dt"].float()), dict(conv_w=d["conv_w"][:-1]),
                   dict(conv_state=d["conv_state"][:3]), dict(state=d["state"][:, :1]), dict(D=d["D"][:1]),
                   dict(state_indices=torch.zeros(3, dtype=torch.int32, device="cuda")),
                   dict(state_indices=torch.zeros(4, dtype=torch.int64, device="cuda")),
                   dict(state=d["state"][:3], conv_state=d["conv_state"][:3]),
                   dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, TypeError, gdn._lib.GdnError)):
            gdn.ssm_decode_step(**{**d, **change})


def test_slots_behind_two_to_the_31(cuda_device):
    H, G, P, N, slots = 32, 1, 128, 128, 4200  # 2^19 states a slot
    d = make(3, 4, H, G, P, N, seed=12)
    small = clone(d)
    C = d["conv_w"].shape[0]
    state = torch.empty(slots, H, N, P, device="cuda")
    conv = torch.empty(slots, C, 3, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([4199, 4097, 0], dtype=torch.int32, device="cuda")
    state[at.long()], conv[at.long()] = d["state"][:3], d["conv_state"][:3]
    y = gdn.ssm_decode_step(**{**d, "state": state, "conv_state": conv, "state_indices": at})
    ref = gdn.ssm_decode_step(**small)
    assert torch.equal(y, ref) and torch.equal(state[at.long()], small["state"][:3])
    assert torch.equal(conv[at.long()], small["conv_state"][:3])


def test_two_calls_at_once(cuda_device):
    sets = [make(64, 64, 8, 2, 64, 128, seed=s) for s in (21, 22)]
    refs = [clone(d) for d in sets]
    for r in refs:
        r["y"] = [gdn.ssm_decode_step(**{k: v for k, v in r.items() if k != "y"}) for _ in range(4)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for k, d in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                got[k].append(gdn.ssm_decode_step(**d))
    torch.cuda.synchronize()
    for k, d in enumerate(sets):
        assert all(torch.equal(a, b) for a, b in zip(got[k], refs[k]["y"]))
        assert torch.equal(d["state"], refs[k]["state"]) and torch.equal(d["conv_state"], refs[k]["conv_state"])


@pytest.mark.parametrize("n", [5, 200])
def test_a_batch_of_padding_is_done_when_its_call_is(cuda_device, n):
    # what comes next in the stream may name live slots in the same tensor: none of them is touched
    d = make(n, n, 2, 1, 64, 64, seed=31)
    idx = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    live = torch.arange(n, dtype=torch.int32, device="cuda")
    before = clone(d)
    for _ in range(50):
        y = gdn.ssm_decode_step(**d, state_indices=idx)
        idx.copy_(live)
        assert not y.any()
        idx.fill_(-1)
    assert torch.equal(d["state"], before["state"]) and torch.equal(d["conv_state"], before["conv_state"])
    assert gdn.device_status() == 0


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("n", [64, 67, 130])
def test_a_decode_batch(cuda_device, n, W, bias):
    # from 64 requests the convolution takes 16-byte accesses, where rows start on 16 bytes: against the
    # definition, and bit for bit what it is on rows that do not (the taps add up in the same order)
    slots = n + 9
    d = make(n, slots, 4, 2, 32, 32, W, seed=n + W, bias=bias, wide=4)
    assert d["row"].data_ptr() % 16 == 0 and d["row"].stride(0) % 8 == 0
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    idx[[0, 5, n - 2]] = -1
    idx[[9, n - 1]] = torch.tensor([slots, 1 << 30], dtype=torch.int32)
    d["state_indices"] = idx.cuda()
    before = clone(d)
    d["y"] = gdn.ssm_decode_step(**d)
    assert gdn.device_status() == 1 and gdn.device_status() == 0
    assert not d["y"][[0, 5, 9, n - 2, n - 1]].any()
    odd = clone(before)
    odd["row"] = torch.nn.functional.pad(before["row"], (1, 0))[:, 1:]
    assert odd["row"].data_ptr() % 16 != 0
    y = gdn.ssm_decode_step(**odd)
    assert gdn.device_status() == 1
    assert torch.equal(y, d["y"]) and torch.equal(odd["state"], d["state"])
    assert torch.equal(odd["conv_state"], d["conv_state"])
    before["state_indices"] = torch.where(idx >= slots, -1, idx).cuda()
    check(d, before)


def test_a_decode_batch_without_activation_or_slots(cuda_device):
    d = make(70, 70, 2, 1, 64, 64, seed=14, wide=6)
    assert d["row"].data_ptr() % 16 == 0 and d["row"].stride(0) % 8 == 0
    before = clone(d)
    y = gdn.ssm_decode_step(**d, activation=False)
    ry, rs, rc, ym, sm = (torch.from_numpy(t) for t in layer.ssm_decode_step(**before, activation=False))
    assert ((y.cpu().double() - ry).abs() <= 2.0 ** -8 * ry.abs() + (96 + 64) * E * ym).all()
    assert ((d["state"].cpu().double() - rs).abs() <= 64 * E * sm).all()
    assert torch.equal(d["conv_state"].cpu().double(), rc)
