"""sv_shape_logits against the CPU oracle (fp64).

Bound of a touched logit, from the arithmetic: the reciprocal of the repetition
penalty and the product with it, the product and sum of the other penalties,
the bias's addition to those and their addition to the logit round to fp32
once each, so six halves of a step, 6 * 2^-24 of the sum of the absolute values
that are added up.  Below 2^-126 fp32 has steps of 2^-149 whatever the value
(a product of 1e-30 and 2^-126 is 0), so half a step there is 2^-150: six of
those are added, which is what a subnormal result can be off by.  Untouched logits are equal to the input,
barred ones are -inf.
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


def _bits(let):
    """bool [n][V] -> int32 words [n][ceil(V / 32)], bits past V set."""
    n, V = let.shape
    W = -(-V // 32)
    full = np.ones((n, W * 32), bool)
    full[:, :V] = let
    return (full.reshape(n, W, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(
        -1).astype(np.uint32).view(np.int32)


class Case:
    def __init__(self, rows, V, dtype=torch.float32, tree=False, pad=0, hist=(0, 50), pen=True,
                 bias=0, masks=None, seed=0, behind=0, few=False):
        rng = np.random.default_rng(seed)
        self.V, self.rng = V, rng
        R = len(rows)
        self.cu = np.zeros(R + 1, np.int32)
        self.cu[1:] = np.cumsum(rows)
        self.N = int(self.cu[-1]) + behind
        self.max_rows = int(max(rows))
        up = [-1 if j == 0 else int(rng.integers(0, j)) if tree else j - 1 for n in rows for j in range(n)]
        self.parent = np.array(up + [0] * behind, np.int32)
        # few distinct tokens: paths and histories repeat them
        word = lambda *n: rng.integers(0, min(V, 7) if few else V, n).astype(np.int32)  # noqa: E731
        self.tokens = word(self.N)
        self.logits = torch.from_numpy(rng.standard_normal((self.N, V + pad)).astype(np.float32) * 3).to(dtype)
        self.kw = {}
        if pen:
            n = rng.integers(hist[0], hist[1] + 1, R).astype(np.int32)
            self.kw = dict(history=word(R, max(1, hist[1])), history_len=n,
                           prompt_len=(n * rng.random(R)).astype(np.int32),
                           repetition=(1 + rng.random(R)).astype(np.float32),
                           frequency=rng.standard_normal(R).astype(np.float32),
                           presence=rng.standard_normal(R).astype(np.float32))
        if bias:
            n = rng.integers(0, bias + 1, R)
            self.kw.update(bias_begin=np.concatenate([[0], np.cumsum(n)]).astype(np.int32),
                           bias_token=word(int(n.sum()) + 1),
                           bias_value=rng.standard_normal(int(n.sum()) + 1).astype(np.float32))
        if masks is not None:
            M = max(1, self.N // 2)
            let = rng.random((M, V)) < masks
            let[np.arange(M), rng.integers(0, V, M)] = True
            self.kw.update(mask=_bits(let), mask_row=rng.integers(-1, M, self.N).astype(np.int32))
        self.windows = {}

    def bind(self, out=None, **over):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        kw = {k: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()
              for k, v in self.kw.items()}
        kw.update(over.pop("rules", {}))
        self.x = self.logits.cuda()[:, :self.V]
        self.out = torch.full((self.N, self.V), 55.0, device="cuda") if out is None else out
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        b = api.Batch(i32(self.cu), i32(self.parent), i32(self.tokens), self.max_rows,
                      **{k: i32(v) for k, v in self.windows.items()})
        a = dict(batch=b, logits=self.x, rules=api.LogitRules(**kw), out=self.out, dev_status=self.status)
        a.update(over)
        return api.bind_shape_logits(**a)

    def want(self):
        x = self.logits[:, :self.V].float().double().numpy()
        return edges.shape_logits(self.cu, self.parent, self.tokens, x, **self.kw)

    def check(self, status=0, rows=None, left=()):
        torch.cuda.synchronize()
        assert self.status.item() == status
        got = self.out.cpu().double().numpy()
        want, mag = self.want()
        x = self.logits[:, :self.V].float().double().numpy()
        rows = np.arange(int(self.cu[-1])) if rows is None else rows
        rest = np.setdiff1d(np.arange(self.N), rows)
        assert (got[rest] == 55.0).all()  # rows that are nobody's or outside
        g, w, m, x = got[rows], want[rows], mag[rows], x[rows]
        assert np.array_equal(np.isnan(g), np.isnan(w))
        fixed = ~np.isfinite(w) | (w == x)
        same = (g == w) | np.isnan(w)
        assert same[fixed & ((w == x) | np.isinf(w))].all()
        with np.errstate(invalid="ignore"):  # of equal infinities
            d = np.abs(np.where(np.isfinite(w), g - w, 0))
        assert (d <= 6 * 2.0 ** -24 * np.where(np.isfinite(m), m, 0) + 6 * 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,pad", [(1, 0), (7, 2), (32, 0), (257, 0), (4096, 0), (4100, 4), (4101, 0),
                                   (8192, 61), (12289, 3), (50257, 47)])
@pytest.mark.parametrize("tree", [False, True])
def test_vocabularies_and_layouts(V, pad, dtype, tree):
    rows = [1, 5, 9, 2] if V > 10000 else [1, 5, 33, 2, 8, 8, 70]
    c = Case(rows, V, dtype, tree, pad, bias=9, masks=0.5, seed=V, few=V < 300)
    c.bind()()
    c.check()


@pytest.mark.parametrize("parts", ["none", "pen", "bias", "mask", "pen bias", "pen mask", "bias mask"])
@pytest.mark.parametrize("V", [4000, 1003])
def test_each_part_alone(parts, V):
    c = Case([3, 1, 17], V, tree=True, pen="pen" in parts, bias=40 if "bias" in parts else 0,
             masks=0.1 if "mask" in parts else None, seed=3)
    c.bind()()
    c.check()


@pytest.mark.parametrize("part", ["repetition", "frequency", "presence"])
def test_each_penalty_alone(part):
    c = Case([4, 6], 900, few=True)
    for k in ("repetition", "frequency", "presence"):
        if k != part:
            c.kw[k] = None
    c.bind()()
    c.check()


def test_without_history_the_path_still_counts():
    c = Case([9, 5], 500, tree=True, few=True)
    for k in ("history", "history_len", "prompt_len"):
        c.kw[k] = None
    c.bind()()
    c.check()


def test_all_history_is_prompt_or_none_of_it():
    c = Case([4, 4, 4], 600, hist=(40, 40), few=True)
    c.kw["prompt_len"] = c.kw["history_len"].copy()
    c.bind()()
    c.check()
    c.kw["prompt_len"] = None
    c.bind()()
    c.check()


def test_long_histories_and_long_chains_of_one_token():
    c = Case([128, 1, 100], 9000, hist=(20000, 40001), few=True)
    c.bind()()
    c.check()


def test_one_full_tree_whose_paths_share_tokens():
    c = Case([128], 5000, tree=True, few=True, masks=0.7)
    c.bind()()
    c.check()


def test_many_requests_in_one_group_of_rows():
    c = Case([1] * 333, 700, bias=5, masks=0.4, few=True)
    c.bind()()
    c.check()


def test_neutral_parameters_change_nothing():
    c = Case([3, 3], 4096)
    c.kw["repetition"][:] = 1
    c.kw["frequency"][:] = c.kw["presence"][:] = 0
    c.bind()()
    c.check()
    assert torch.equal(c.out, c.x)


def test_tokens_outside_the_vocabulary_are_ignored():
    c = Case([4, 7], 300, bias=30, hist=(30, 60))
    c.kw["history"][:, ::3] = -1
    c.kw["history"][:, 1::7] = 300
    c.kw["bias_token"][::2] = 1 << 30
    c.tokens[2], c.tokens[6] = -5, 300
    c.bind()()
    c.check()


def test_a_token_biased_twice_takes_its_first_entry():
    c = Case([5], 64, bias=200, few=True)
    c.bind()()
    c.check()


def test_infinities_and_nan():
    c = Case([2, 3], 256, masks=0.5, bias=20)
    x = c.logits
    x[:, 3::17] = -np.inf
    x[:, 5::23] = np.inf
    x[0, 7::11] = np.nan
    x[:, 9] = torch.finfo(torch.float32).min
    c.kw["bias_value"][::5] = -np.inf
    c.bind()()
    torch.cuda.synchronize()
    got = c.out.cpu().double().numpy()
    want, mag = c.want()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    ok = np.isfinite(want) & (np.abs(want) < 1e38)
    assert (np.abs(got[ok] - want[ok]) <= 6 * 2.0 ** -24 * mag[ok]).all()


@pytest.mark.parametrize("V", [64, 4097, 9000])
def test_masks_that_let_little_or_nothing_through(V):
    c = Case([3, 2, 4], V, masks=0.5)
    m = c.kw["mask"]
    m[:] = 0
    for k in range(1, len(m)):
        m[k, (V - 1) // 32] = 1 << ((V - 1) % 32) if (V - 1) % 32 < 31 else -(1 << 31)
    c.kw["mask_row"] = np.array([1, 2, 3, -1, 1, 1, 2, 3, 2], np.int32)
    c.bind()()
    c.check()
    c.kw["mask_row"][4] = 0  # lets nothing through: not applied
    c.bind()()
    c.check(status=edges.EMPTY_MASK)
    if V % 32:  # only bits that name no token
        m[0, V // 32] = np.int32(-1) << (V % 32)
        c.bind()()
        c.check(status=edges.EMPTY_MASK)


def test_mask_rows_by_position_and_out_of_range():
    c = Case([3, 2], 100, masks=0.3)
    c.kw["mask"] = _bits(np.random.default_rng(0).random((5, 100)) < 0.3)
    c.kw["mask_row"] = None
    c.bind()()
    c.check()
    c.kw["mask_row"] = np.array([0, 5, 1, -2, 4], np.int32)
    c.bind()()
    c.kw["mask_row"] = np.array([0, -1, 1, -1, 4], np.int32)
    c.check(status=edges.BAD_PARAM)


@pytest.mark.parametrize("rho", [2.0 ** -126, 2.0 ** 126, 1e-3, 1e3])
def test_the_repetition_penalty_over_its_range(rho):
    c = Case([4, 4], 400, few=True, hist=(30, 50))
    c.kw["repetition"][:] = rho
    c.kw["frequency"][:] = c.kw["presence"][:] = 0
    x = c.logits
    x[:, :7] = torch.tensor([-2.0, 0.0, 1.0, 3e-38 if rho < 1 else 3.0, 2.0 ** -10, -0.0, -1e-30])
    if rho < 1e-6:  # what overflows is infinite
        x[:, [2, 4]] = 0.0
    if rho > 1e6:
        x[:, 0] = -1e-38
    c.bind()()
    c.check()


def test_without_a_status_word_findings_are_dropped():
    c = Case([3, 4, 5], 500)
    c.kw["repetition"][1] = -1
    c.bind(dev_status=None)()
    torch.cuda.synchronize()
    assert (c.out[3:7] == 55).all() and (c.out[:3] != 55).any() and c.status.item() == 0


def test_windows_and_padding_rows():
    c = Case([5, 9, 1, 12], 1000, tree=False, masks=0.6, behind=6)
    c.windows = dict(row_begin=[1, 0, 1, 4], row_end=[3, 9, 1, 12], verify_len=[9, 3, 9, 6])
    c.bind()()
    rows = [1, 2] + list(range(5, 9)) + [15 + j for j in range(4, 7)]
    c.check(rows=np.array(rows))


@pytest.mark.parametrize("spoil,status", [
    (lambda c: c.kw["repetition"].__setitem__(1, 0.0), edges.BAD_PARAM),
    (lambda c: c.kw["repetition"].__setitem__(1, -1.0), edges.BAD_PARAM),
    (lambda c: c.kw["repetition"].__setitem__(1, 1e-39), edges.BAD_PARAM),
    (lambda c: c.kw["repetition"].__setitem__(1, 2e38), edges.BAD_PARAM),
    (lambda c: c.kw["repetition"].__setitem__(1, np.nan), edges.BAD_PARAM),
    (lambda c: c.kw["repetition"].__setitem__(1, np.inf), edges.BAD_PARAM),
    (lambda c: c.kw["frequency"].__setitem__(1, np.nan), edges.BAD_PARAM),
    (lambda c: c.kw["presence"].__setitem__(1, -np.inf), edges.BAD_PARAM),
    (lambda c: c.kw["history_len"].__setitem__(1, 51), edges.BAD_LENGTH),
    (lambda c: c.kw["history_len"].__setitem__(1, -1), edges.BAD_LENGTH),
    (lambda c: c.kw["prompt_len"].__setitem__(1, c.kw["history_len"][1] + 1), edges.BAD_LENGTH),
    (lambda c: c.kw["prompt_len"].__setitem__(1, -1), edges.BAD_LENGTH),
    (lambda c: c.parent.__setitem__(6, 3), edges.BAD_PARENT),
    (lambda c: c.parent.__setitem__(3, 0), edges.BAD_PARENT),
])
def test_a_bad_request_is_left_alone(spoil, status):
    c = Case([3, 4, 5], 500, tree=True)
    good, parent = {k: v.copy() for k, v in c.kw.items()}, c.parent.copy()
    spoil(c)
    c.bind()()
    c.kw, c.parent = good, parent
    c.check(status=status, rows=np.r_[0:3, 7:12])


def test_bad_bias_ranges_are_left_alone():
    c = Case([2, 2, 2], 100, bias=5)
    n = c.kw["bias_token"].size
    good = {k: v.copy() for k, v in c.kw.items()}
    c.kw["bias_begin"] = np.array([0, 3, n + 1, n], np.int32)
    c.bind()()
    c.kw["bias_begin"] = np.array([0, 3, 3, 3], np.int32)
    c.check(status=edges.BAD_PARAM, rows=np.r_[0:2])
    del good


def test_in_place_and_apart_agree():
    for V in (4096, 4099):
        c = Case([5, 6], V, bias=9, masks=0.5, tree=True)
        c.bind()()
        c.check()
        x = c.x.contiguous().clone()
        c.bind(out=x, logits=x)()
        first = c.out
        c.bind()()
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("masks", [None, 0.5])
@pytest.mark.parametrize("V", [4096, 9001])
def test_single_rows_in_place(V, masks):
    c = Case([1] * 40, V, bias=9, masks=masks, few=V < 5000)
    x = c.logits.cuda()
    c.bind(out=x, logits=x)()
    c.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(620, 8192), (640, 5003), (310, 8196), (310, 8195), (160, 24581),
                                 (100, 50257), (90, 50260)])
@pytest.mark.parametrize("parts", ["pen", "pen bias mask", "bias mask"])
def test_many_single_rows(R, V, dtype, parts):
    c = Case([1] * R, V, dtype, pad=R % 3, hist=(0, 600), pen="pen" in parts,
             bias=60 if "bias" in parts else 0, masks=0.3 if "mask" in parts else None, seed=V,
             few=R == 310, behind=2)
    c.bind()()
    c.check()


def test_many_single_rows_in_place_and_spoilt():
    c = Case([1] * 640, 4003, bias=20, masks=0.5, hist=(0, 90))
    c.bind()()
    c.check()
    first, x = c.out, c.x.contiguous().clone()
    c.bind(out=x, logits=x)()
    torch.cuda.synchronize()
    assert torch.equal(first, x)
    good = {k: v.copy() for k, v in c.kw.items()}
    c.kw["history_len"][639] = 91
    c.kw["repetition"][7] = 0.0
    c.bind()()
    c.kw = good
    c.check(status=edges.BAD_LENGTH | edges.BAD_PARAM, rows=np.r_[0:7, 8:639])


@pytest.mark.parametrize("n", [65533, 65534, 65535, 70000])
def test_single_rows_with_long_lists_of_biases(n):
    # a token's only entry may be the list's last, whatever the list's length
    c = Case([1] * 620, 8000, hist=(0, 20))
    token = c.rng.integers(0, 7000, n).astype(np.int32)
    token[-1] = 7999
    begin = np.full(621, n, np.int32)
    begin[0] = 0
    c.kw.update(bias_begin=begin, bias_token=token,
                bias_value=c.rng.standard_normal(n).astype(np.float32))
    c.bind()()
    c.check()


def test_misaligned_rows_and_outputs():
    c = Case([5, 6], 4096, bias=9, masks=0.5)
    wide = torch.zeros(11 * 4096 + 4, device="cuda")
    out = wide[1:-3].view(11, 4096)
    out.fill_(55)
    c.bind(out=out)()
    c.check()
    assert wide[0] == 0 and (wide[-3:] == 0).all()
    big = torch.zeros(11, 4099, device="cuda")
    big[:, 2:4098] = c.x
    c.bind(logits=big[:, 2:4098])()
    c.check()


def test_stream_and_graph_and_repeats():
    c = Case([9] * 30, 5000, tree=True, bias=20, masks=0.5, few=True)
    call = c.bind()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(s)
    c.check()
    first = c.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        c.out.fill_(55)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first)


def test_two_batches_at_once_on_two_streams():
    cases = [Case([9] * 20, 9000, tree=True, bias=20, masks=0.5, few=True, seed=k) for k in range(2)]
    calls = [c.bind() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for call, s in zip(calls, streams):
            call(s)
    for c in cases:
        c.check()


def test_more_logits_than_32_bits_count():
    # 2.2 billion logits: the last rows' offsets pass 2^31 and 2^32 bytes
    V, N = 151936, 14500
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = torch.empty(N, V, device="cuda")
    cu = torch.arange(0, N + 1, 5, dtype=torch.int32, device="cuda")
    parent = (torch.arange(N, device="cuda") % 5 - 1).int()
    R = N // 5
    b = api.Batch(cu, parent, torch.full((N,), 7, dtype=torch.int32, device="cuda"), 5)
    one = torch.ones(R, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sv_shape_logits(b, x, api.LogitRules(presence=one, frequency=one), out, st)
    assert st.item() == 0
    j = torch.arange(N, device="cuda") % 5
    want = x[:, 7].float() - (j + (j > 0)).float()  # the path's drafts are all token 7
    assert ((out[:, 7] - want).abs() <= 2.0 ** -21 * (x[:, 7].float().abs() + 5)).all()
    out[:, 7] = x[:, 7].float()
    for r in range(0, N, 2900):
        assert torch.equal(out[r:r + 2900], x[r:r + 2900].float())


@pytest.mark.parametrize("over,words", [
    (lambda c: dict(logits=c.logits.cuda().half()), "float32 or bfloat16"),
    (lambda c: dict(logits=c.logits.cuda()[:3]), "must be"),
    (lambda c: dict(logits=c.logits.cuda()[:, :50]), "must be"),
    (lambda c: dict(logits=c.logits.t().contiguous().cuda().t()), "dense"),
    (lambda c: dict(logits=c.logits), "tensors of one call"),
    (lambda c: dict(rules=dict(repetition=torch.ones(1, device="cuda"))), "at least"),
    (lambda c: dict(rules=dict(frequency=torch.ones(2, device="cuda").double())), "float32"),
    (lambda c: dict(rules=dict(history=torch.zeros(50, dtype=torch.int32, device="cuda"))), "history must be"),
])
def test_binding_refuses(over, words):
    c = Case([3, 4], 100)
    with pytest.raises(SpecVerifyError, match=words):
        c.bind(**over(c))


def test_call_refuses():
    c = Case([3, 4], 100, masks=0.5)
    z = torch.zeros(8, 100, device="cuda")
    for over in (dict(rules=dict(mask=torch.zeros(9, 3, dtype=torch.int32, device="cuda"))),  # too few words
                 dict(rules=dict(mask_row=None)),                                             # fewer masks than rows
                 dict(rules=dict(history_len=None)),
                 dict(logits=z[:7], out=z[1:])):                                              # overlap
        with pytest.raises(SpecVerifyError):
            c.bind(**over)()
