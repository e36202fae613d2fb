"""sv_stage_qkv against the CPU oracle (fp64).

Bound of a normed and rotated element, from the arithmetic: the mean of at
most 128 squares is off by 2^-17 of itself at worst (128 fp32 roundings), its
root by half of that, and the root, the two products of the norm, cosine and
sine (angle within 2^-23 rad, one or two units of the last place), the two
products and the sum of the rotation by a few 2^-24 each: in all below 2^-16
of |a| + |b|.  The store rounds to bf16: half a step, 2^-8 of the value.
Copied elements (V, K and Q without norm and rotation) are equal.
"""

import numpy as np
import pytest
import torch

from oracle import edges
from speculative_decoding_verification_padding_gb300 import api, build
from speculative_decoding_verification_padding_gb300._native import SpecVerifyError

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


class Case:
    def __init__(self, rows, heads, kv_heads, dim, rotary=None, axes=1, interleaved=False,
                 norm=True, far=5000, scale=1.0, packed=True, skip=0, seed=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.K, self.D, self.N = heads, kv_heads, dim, rows
        self.rd = dim if rotary is None else rotary
        x = (torch.randn(rows, (heads + 2 * kv_heads) * dim, generator=g) * spread).bfloat16()
        q, k, v = (t if packed else t.clone().contiguous()
                   for t in x.cuda().split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
        self.q, self.k, self.v = (t.unflatten(1, (-1, dim)) for t in (q, k, v))
        blocks = -(-rows // 16) + 3
        self.slots = torch.randperm(blocks * 16, generator=g)[:rows].int()
        if skip:
            self.slots[torch.randperm(rows, generator=g)[:skip]] = -1
        self.pos = torch.randint(0, far + 1, (axes, rows), generator=g).int()
        half = self.rd // 2
        self.freq = (10000.0 ** (-torch.arange(half).double() / max(half, 1))).float()
        self.axis = torch.randint(0, axes, (half,), generator=g).int() if axes > 1 else None
        self.inter, self.scale = interleaved, scale
        self.qw, self.kw = ((1 + 0.3 * torch.randn(dim, generator=g)).float() if norm else None
                            for _ in range(2))
        self.eps = 1e-5
        self.kc = torch.randn(blocks, kv_heads, 16, dim, generator=g).bfloat16()
        self.vc = torch.randn(blocks, kv_heads, 16, dim, generator=g).bfloat16()
        self.out0 = torch.full((rows, heads, dim), 77.0, dtype=torch.bfloat16)

    def bind(self, **over):
        cu = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.dev = dict(kc=self.kc.cuda(), vc=self.vc.cuda(), out=self.out0.cuda(),
                        status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        z = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        rotary = api.Rotary(cu(self.freq), self.rd, cu(self.axis), self.inter, self.scale) if self.rd else None
        pos = self.pos if self.axis is not None else self.pos[0]
        a = dict(kv=api.PagedKV(self.dev["kc"], self.dev["vc"], z, z[0]), q=self.q, k=self.k, v=self.v,
                 slots=cu(self.slots), positions=cu(pos) if self.rd else None, rotary=rotary,
                 q_out=self.dev["out"], q_weight=cu(self.qw), k_weight=cu(self.kw), eps=self.eps,
                 dev_status=self.dev["status"])
        a.update(over)
        return api.bind_stage_qkv(**a)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert self.dev["status"].item() == status
        f64 = lambda t: t.float().cpu().double().numpy()  # noqa: E731
        live = (self.slots >= 0) & (self.slots < self.kc.shape[0] * 16)
        live = live.numpy()
        block, off = (self.slots.numpy() // 16)[live], (self.slots.numpy() % 16)[live]
        want_q, tol_q = f64(self.out0), np.zeros(self.out0.shape)
        want_k, tol_k = f64(self.kc), np.zeros(self.kc.shape)
        want_v = f64(self.vc)
        for x, w, want, tol, put in ((self.q, self.qw, want_q, tol_q, lambda a, y: a.__setitem__(live, y)),
                                     (self.k, self.kw, want_k, tol_k,
                                      lambda a, y: a.__setitem__((block, slice(None), off), y))):
            w = None if w is None else w.numpy()
            y, mag = edges.stage(f64(x), w, self.eps, self.pos.numpy(), self.freq.numpy(), self.rd,
                                 None if self.axis is None else self.axis.numpy(), self.inter, self.scale)
            t = 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * mag
            if w is None:
                t[..., self.rd:] = 0
            put(want, y[live])
            put(tol, t[live])
        want_v[block, :, off] = f64(self.v)[live]
        for got, want, tol in ((self.dev["out"], want_q, tol_q), (self.dev["kc"], want_k, tol_k)):
            d = np.abs(f64(got) - want)
            assert (d <= tol).all(), float((d - tol).max())
        assert np.array_equal(f64(self.dev["vc"]), want_v)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 2), (5, 5), (14, 2), (32, 4), (64, 8), (96, 32)])
@pytest.mark.parametrize("rows", [1, 6, 333])
def test_head_layouts_and_rows(rows, heads, kv_heads, dim):
    c = Case(rows, heads, kv_heads, dim, seed=rows + heads)
    c.bind()()
    c.check()


@pytest.mark.parametrize("rows,heads,kv_heads,dim", [(3, 200, 8, 128), (150, 300, 40, 128), (2, 1000, 1, 64),
                                                     (1300, 130, 3, 128), (1400, 90, 12, 64)])
def test_rows_wider_than_a_block_holds_at_once(rows, heads, kv_heads, dim):
    c = Case(rows, heads, kv_heads, dim, rotary=dim // 2, seed=heads)
    c.bind()()
    c.check()


@pytest.mark.parametrize("dim,rotary", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 0), (128, 48), (128, 112),
                                        (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_partial_rotation_of_many_rows(dim, rotary, interleaved):
    c = Case(5001, 5, 2, dim, rotary, axes=3 if rotary else 1, interleaved=interleaved, skip=3, seed=rotary)
    c.bind()()
    c.check()


@pytest.mark.parametrize("rows,heads,kv_heads,dim,skip", [
    (2600, 64, 8, 128, 0), (2600, 64, 8, 128, 2500), (2433, 21, 2, 128, 7), (4300, 33, 8, 64, 40), (4865, 3, 1, 64, 0),
    (4864, 4, 1, 64, 9), (5100, 10, 3, 64, 5000), (1700, 70, 1, 128, 100)])
def test_many_rows_that_take_turns(rows, heads, kv_heads, dim, skip):
    c = Case(rows, heads, kv_heads, dim, axes=2, skip=skip, seed=rows)
    c.bind()()
    c.check()


@pytest.mark.parametrize("dim,rotary", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 0), (128, 32),
                                        (128, 80), (128, 96), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_partial_rotation(dim, rotary, interleaved, norm):
    c = Case(19, 6, 2, dim, rotary, interleaved=interleaved, norm=norm)
    c.bind()()
    c.check()


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_several_position_axes(axes, interleaved):
    c = Case(77, 4, 1, 128, axes=axes, interleaved=interleaved, scale=1.25)
    c.bind()()
    c.check()


@pytest.mark.parametrize("far", [0, 1 << 20, (1 << 31) - 1])
def test_far_and_negative_positions(far):
    # the fp64 oracle's own angle is good to 2^-53 of it, 2^-22 rad at 2^31
    c = Case(200, 2, 1, 128, far=far)
    c.pos[0, ::3] = far
    c.pos[0, 1::3] = -far
    c.bind()()
    c.check()


def test_many_rows_more_than_one_wave():
    c = Case(5003, 3, 1, 64, skip=100)
    c.bind()()
    c.check()


@pytest.mark.parametrize("spread", [1e-20, 1e-4, 1e4, 1e15])
def test_small_and_large_heads(spread):
    # eps rules for tiny heads; squares of 1e15 stay finite in fp32
    c = Case(9, 4, 2, 128, spread=spread)
    c.bind()()
    c.check()


def test_zero_heads_stay_zero():
    c = Case(4, 4, 2, 64)
    c.q, c.k = torch.zeros_like(c.q), torch.zeros_like(c.k)
    c.bind()()
    c.check()
    assert (c.dev["out"] == 0).all()


def test_skipped_and_bad_slots():
    c = Case(64, 4, 2, 64, skip=20)
    c.slots[3] = c.kc.shape[0] * 16
    c.slots[40] = -2
    c.slots[63] = (1 << 31) - 1
    c.bind()()
    c.check(status=edges.BAD_SLOT)


def test_bad_axis_reads_axis_zero():
    c = Case(10, 2, 1, 64, axes=2)
    good = c.axis.clone()
    c.axis[3], c.axis[9] = 2, -1
    c.bind()()
    c.axis = good
    c.axis[3] = c.axis[9] = 0
    c.check(status=edges.BAD_PARAM)


def test_in_place_rows_apart_and_dense():
    a, b = Case(50, 8, 2, 128, packed=True), Case(50, 8, 2, 128, packed=False)
    assert a.q.stride(0) != b.q.stride(0) and not a.q.is_contiguous()
    a.bind()()
    keep = b.q.clone()
    b.bind(q_out=b.q)()  # q turned in place
    torch.cuda.synchronize()
    assert torch.equal(a.dev["out"], b.q) and torch.equal(a.dev["kc"], b.dev["kc"])
    b.q = keep
    a.check()


def test_shared_position_for_every_axis():
    c = Case(30, 4, 2, 64, axes=3)
    c.pos[1:] = c.pos[0]
    call = c.bind(positions=c.pos[0].cuda())
    call()
    c.check()


def test_the_c_call_with_one_position_on_three_axes():
    import ctypes
    from speculative_decoding_verification_padding_gb300 import _native as N
    c = Case(30, 4, 2, 64, axes=3)
    c.pos[1:] = c.pos[0]
    c.bind()
    keep = [t.cuda() for t in (c.slots, c.pos[0], c.freq, c.axis, c.qw, c.kw)]
    slots, pos, freq, axis, qw, kw = (t.data_ptr() for t in keep)
    d = c.dev
    kv = N.SvPagedKV(d["kc"].data_ptr(), d["vc"].data_ptr(), c.kc.shape[0], 16, 2, 64, None, 0, None)
    rot = N.SvRotary(freq, 64, 0, 3, axis, 1.0)
    step = c.q.stride(0)
    assert N.lib().sv_stage_qkv(ctypes.byref(kv), 30, c.q.data_ptr(), step, c.k.data_ptr(), step, c.v.data_ptr(), step,
                                4, slots, pos, 0, ctypes.byref(rot), qw, kw, c.eps, d["out"].data_ptr(), None,
                                torch.cuda.current_stream().cuda_stream) == N.SV_OK
    c.check()


def test_far_blocks_and_two_streams_at_once():
    # cache slots whose element offsets pass 2^31, and two calls side by side
    K, D, blocks = 8, 128, 140000
    kc = torch.zeros(blocks, K, 16, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    c = Case(40, 16, K, D)
    d = Case(40, 16, K, D, seed=1)
    z = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    calls = []
    for k, case in enumerate((c, d)):
        case.slots = (torch.arange(40) * 2 + k + (blocks - 5) * 16).int()
        calls.append(case.bind(kv=api.PagedKV(kc, vc, z, z[0])))
    torch.cuda.synchronize()
    for call in calls:
        call(torch.cuda.Stream())
    torch.cuda.synchronize()
    for case in (c, d):
        small = {"kc": case.kc, "vc": case.vc}
        at = case.slots.long().cuda()
        for name, big in (("kc", kc), ("vc", vc)):
            got = big[at // 16, :, at % 16]
            # the same rows into a small cache, whose result test_head_layouts checks
            assert (got.float().abs().sum((1, 2)) > 0).all()
            small[name] = got
        case.slots = torch.arange(40).int()
        case.bind()()
        torch.cuda.synchronize()
        at = case.slots.long().cuda()
        assert torch.equal(case.dev["kc"][at // 16, :, at % 16], small["kc"])
        assert torch.equal(case.dev["vc"][at // 16, :, at % 16], small["vc"])
    assert kc[: blocks - 5].abs().max() == 0


def test_stream_and_graph():
    c = Case(21, 8, 2, 64)
    s = torch.cuda.Stream()
    call = c.bind()
    torch.cuda.synchronize()
    call(s)
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    c.dev["out"].fill_(77)
    c.dev["kc"].copy_(c.kc)
    c.dev["vc"].copy_(c.vc)
    g.replay()
    c.check()


@pytest.mark.parametrize("over,words", [
    (lambda c: dict(q=c.q[:, :, ::2]), "q must be"),
    (lambda c: dict(q=torch.cat([c.q, c.q], 2)[:, :, ::2]), "dense"),
    (lambda c: dict(k=c.k[:, :1]), "k must be"),
    (lambda c: dict(q=c.q.half()), "bfloat16"),
    (lambda c: dict(slots=c.slots[:3].cuda()), "slots must be"),
    (lambda c: dict(slots=c.slots), "tensors of one call"),
    (lambda c: dict(positions=c.pos[0][:4].cuda()), "positions must be"),
    (lambda c: dict(q_weight=torch.ones(3, device="cuda")), "at least"),
    (lambda c: dict(rotary=api.Rotary(c.freq.cuda()[:4], c.rd)), "at least"),
])
def test_binding_refuses(over, words):
    c = Case(9, 4, 2, 64)
    with pytest.raises(SpecVerifyError, match=words):
        c.bind(**over(c))


@pytest.mark.parametrize("over", [
    lambda c: dict(rotary=api.Rotary(c.freq.cuda(), 24)),        # not a multiple of 16
    lambda c: dict(rotary=api.Rotary(c.freq.cuda(), -16)),
    lambda c: dict(positions=None),
    lambda c: dict(positions=c.pos.repeat(2, 1).cuda()),          # two axes, no freq_axis
    lambda c: dict(eps=-1.0),
    lambda c: dict(eps=float("nan")),
    lambda c: dict(q_weight=torch.ones(65, device="cuda")[1:]),   # 4 bytes off
    lambda c: dict(q_out=torch.empty(9 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[4:-4].view(9, 4, 64)),
])
def test_call_refuses(over):
    c = Case(9, 4, 2, 64)
    call = c.bind(**over(c))
    with pytest.raises(SpecVerifyError):
        call()
    torch.cuda.synchronize()
    assert torch.equal(c.dev["kc"].cpu(), c.kc)


def test_call_refuses_overlap():
    c = Case(9, 4, 2, 64)
    wide = torch.zeros(10, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(SpecVerifyError):
        c.bind(q=wide[:9], q_out=wide[1:])()
    with pytest.raises(SpecVerifyError):
        c.bind(k=c.k, q_out=torch.as_strided(c.k, (9, 4, 64), (256, 64, 1)))()
