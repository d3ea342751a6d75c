"""tok_embed and tok_embed_backward against plain loops in 64 bits: every pair
of types, widths and strides that take the ways by eights and by ones, ids
without a row, counts on the device, tokens that come thousands of times, and
the refusals.  The gradient also against differences."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

KINDS = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module")
def env():
    import torch

    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    import exact_bpe_tokenization_utf_gb300 as pkg
    tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    yield torch, pkg, tok
    tok.close()


def _type(torch, kind):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]


def _code(pkg, kind):
    return {"f32": pkg.DTYPE_F32, "f16": pkg.DTYPE_F16, "bf16": pkg.DTYPE_BF16}[kind]


def _half_step(torch, kind):
    return torch.finfo(_type(torch, kind)).eps / 2


def _array(torch, kind, rows, dim, pad, shift, fill=None, seed=0):
    """rows of dim elements, pad apart, from an address `shift` elements past a 16-byte boundary; and all of its memory."""
    store = torch.full((rows * (dim + pad) + shift + 16,), 9.0, dtype=_type(torch, kind), device="cuda")
    a = store[shift:shift + rows * (dim + pad)].view(rows, dim + pad)[:, :dim]
    if fill is None:
        g = torch.Generator(device="cuda").manual_seed(seed)
        a.copy_(torch.randn(rows, dim, generator=g, device="cuda"))
    else:
        a.fill_(fill)
    return a, store


def _ids(seed, n, rows):
    rng = np.random.default_rng(seed)
    ids = np.minimum((rng.random(n) ** 3 * rows).astype(np.int64), rows - 1)
    ids[rng.random(n) < 0.05] = rng.choice([-1, rows, 2**31 - 1, -2**31])
    return ids


class _Call:
    def __init__(self, env, ids, rows, dim, w_kind, o_kind, scale=1.0, count=None, w_pad=0, o_pad=0, shift=0, seed=0, cap=None):
        self.torch, self.pkg, self.tok = env
        torch = self.torch
        self.ids, self.rows, self.dim, self.scale = np.asarray(ids, np.int64), rows, dim, scale
        self.n = len(self.ids)
        self.count = count
        self.used = self.n if count is None else max(0, min(self.n, count))
        self.w_kind, self.o_kind = w_kind, o_kind
        self.d_ids = torch.from_numpy(self.ids.astype(np.int32)).cuda() if self.n else torch.zeros(1, dtype=torch.int32, device="cuda")
        self.d_n = None if count is None else torch.tensor([count], dtype=torch.int64, device="cuda")
        self.w_pad, self.o_pad, self.shift, self.seed = w_pad, o_pad, shift, seed

    def _stream(self):
        return self.torch.cuda.current_stream().cuda_stream

    def forward(self, **other):
        torch = self.torch
        w, _ = _array(torch, self.w_kind, self.rows, self.dim, self.w_pad, self.shift, seed=self.seed)
        out, store = _array(torch, self.o_kind, self.n, self.dim, self.o_pad, self.shift, fill=5.0)
        f = dict(d_ids=self.d_ids.data_ptr(), n=self.n, d_n=None if self.d_n is None else self.d_n.data_ptr(),
                 d_weight=w.data_ptr(), weight_stride=self.dim + self.w_pad, weight_dtype=_code(self.pkg, self.w_kind),
                 n_rows=self.rows, dim=self.dim, scale=self.scale, d_out=out.data_ptr(), out_stride=self.dim + self.o_pad,
                 out_dtype=_code(self.pkg, self.o_kind))
        f.update(other)
        self.tok.embed_device(self.pkg.EmbedArgs(**f), self._stream())
        return w, out, store

    def check_forward(self):
        torch = self.torch
        w, out, store = self.forward()
        there = torch.from_numpy((self.ids[:self.used] >= 0) & (self.ids[:self.used] < self.rows)).cuda()
        at = torch.from_numpy(self.ids[:self.used].clip(0, self.rows - 1)).cuda()
        want = torch.where(there[:, None], w[at].double() * float(np.float32(self.scale)), 0.0)
        got = out[:self.used].double()
        # a 32-bit product, rounded to out's type: one or two roundings
        tol = want.abs() * (2.0**-24 + _half_step(torch, self.o_kind) * (1 + 2.0**-20)) + 2.0**-26
        assert bool(((got - want).abs() <= tol).all())
        assert bool((got[~there] == 0).all())
        assert bool((out[self.used:] == 5).all())
        spare = torch.ones_like(store, dtype=torch.bool)
        spare[self.shift:self.shift + self.n * (self.dim + self.o_pad)].view(self.n, -1)[:, :self.dim] = False
        assert bool((store[spare] == 9).all())

    def backward(self, accumulate=False, start=3.0, work=None, grad=None, into=None, **other):
        torch = self.torch
        if grad is None:
            grad, _ = _array(torch, self.o_kind, max(self.n, 1), self.dim, self.o_pad, self.shift, seed=self.seed + 1)
            grad[self.used:] = float("nan")   # not read
        gw, store = into or _array(torch, self.w_kind, self.rows, self.dim, self.w_pad, self.shift, fill=start)
        size = self.tok.embed_work_bytes(self.n, self.rows, self.dim)
        work = torch.full((size,), 0xee, dtype=torch.uint8, device="cuda") if work is None else work
        f = dict(d_ids=self.d_ids.data_ptr(), n=self.n, d_n=None if self.d_n is None else self.d_n.data_ptr(),
                 n_rows=self.rows, dim=self.dim, scale=self.scale, d_grad_out=grad.data_ptr(),
                 grad_out_stride=self.dim + self.o_pad, grad_out_dtype=_code(self.pkg, self.o_kind),
                 d_grad_weight=gw.data_ptr(), grad_weight_stride=self.dim + self.w_pad,
                 grad_weight_dtype=_code(self.pkg, self.w_kind), accumulate=int(accumulate), d_work=work.data_ptr(),
                 work_bytes=size)
        f.update(other)
        self.tok.embed_backward_device(self.pkg.EmbedGradArgs(**f), self._stream())
        return grad, gw, store

    def check_backward(self, accumulate=False):
        torch = self.torch
        grad, gw, store = self.backward(accumulate)
        ids = torch.from_numpy(self.ids[:self.used]).cuda()
        ok = (ids >= 0) & (ids < self.rows)
        total = torch.zeros(self.rows, self.dim, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(total)
        g = grad[:self.used].double()
        total.index_add_(0, ids[ok], g[ok])
        size.index_add_(0, ids[ok], g[ok].abs())
        times = torch.zeros(self.rows, dtype=torch.int64, device="cuda").index_add_(0, ids[ok], torch.ones_like(ids[ok]))
        scale = float(np.float32(self.scale))
        want = total * scale + (3.0 if accumulate else 0.0)
        # the sum of m numbers in 32 bits, in any order: at most m - 1 roundings of partial sums,
        # none above the sum of the sizes; then a product, perhaps a sum, and the type's rounding
        m = times[:, None].double()
        tol = size * abs(scale) * (m + 2) * 2.0**-24 + want.abs() * (_half_step(torch, self.w_kind) + 2.0**-23) * (1 + 2.0**-8)
        tol += 2.0**-25   # (below the smallest ordinary number of 16 bits, half a step)
        assert bool(((gw.double() - want).abs() <= tol).all())
        rest = gw[times == 0]
        assert bool((rest == (3.0 if accumulate else 0.0)).all())
        spare = torch.ones_like(store, dtype=torch.bool)
        spare[self.shift:self.shift + self.rows * (self.dim + self.w_pad)].view(self.rows, -1)[:, :self.dim] = False
        assert bool((store[spare] == 9).all())
        return gw


@pytest.mark.parametrize("w_kind", KINDS)
@pytest.mark.parametrize("o_kind", KINDS)
def test_types(env, w_kind, o_kind):
    for dim, w_pad, o_pad, shift in ((64, 0, 0, 0), (1032, 8, 16, 8), (257, 0, 3, 1), (64, 1, 0, 0), (7, 2, 2, 3)):
        c = _Call(env, _ids(1, 700, 300), 300, dim, w_kind, o_kind, scale=8.25, w_pad=w_pad, o_pad=o_pad, shift=shift)
        c.check_forward()
        c.check_backward()
        c.check_backward(accumulate=True)


@pytest.mark.parametrize("rows", [1, 2, 31, 33, 2047, 2048, 5000, 100257])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 4096, 4097, 20011])
def test_sizes(env, n, rows):
    dim = 24 if rows * n < 1 << 28 else 8
    c = _Call(env, _ids(n + rows, n, rows), rows, dim, "f32", "bf16", scale=0.5)
    c.check_forward()
    c.check_backward()
    c.check_backward(accumulate=True)


@pytest.mark.parametrize("dim", [1, 8, 255, 256, 264, 1024, 1031, 4096])
def test_widths(env, dim):
    c = _Call(env, _ids(dim, 3000, 800), 800, dim, "bf16", "bf16")
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("count", [-5, 0, 1, 32, 999, 5000, 5001, 10**12])
def test_counts_on_the_device(env, count):
    for dim in (40, 41):
        c = _Call(env, _ids(3, 5000, 400), 400, dim, "f16", "f32", count=count)
        c.check_forward()
        c.check_backward()
        c.check_backward(accumulate=True)


def test_one_id_many_times(env):
    # runs over many chunks and spans; all tokens of one row; none with a row
    for n in (33, 5000, 300007):
        for ids in (np.zeros(n), np.full(n, 77), np.where(np.arange(n) % 3 == 0, 5, 6), np.full(n, -1), np.arange(n) % 2 * 200,
                    np.sort(_ids(n, n, 120)), np.where(np.arange(n) < n // 2, 119, 0)):
            c = _Call(env, ids, 120, 16, "f32", "f32")
            c.check_backward()
            c.check_backward(accumulate=True)


def test_the_largest_vocabulary(env):
    rows = 1 << 20
    ids = np.concatenate([[rows - 1, 0, rows - 1, rows, rows - 2], _ids(5, 30000, rows)])
    c = _Call(env, ids, rows, 8, "bf16", "bf16")
    c.check_forward()
    c.check_backward()


def test_nothing_to_do(env):
    torch, pkg, tok = env
    c = _Call(env, [], 50, 8, "f32", "f32")
    c.forward(d_ids=None, d_weight=None, d_out=None)
    _, gw, _ = c.backward(d_ids=None, d_grad_out=None)
    assert bool((gw == 0).all())
    _, gw, _ = c.backward(accumulate=True, d_ids=None, d_grad_out=None, d_work=None)
    assert bool((gw == 3).all())


def test_infinities_and_nan_stay_in_their_rows(env):
    torch = env[0]
    ids = np.array([4, 2, 4, 9, -1, 2])
    c = _Call(env, ids, 12, 32, "f32", "f32")
    grad = torch.ones(6, 32, device="cuda")
    grad[0, 3], grad[3, 5], grad[4] = float("inf"), float("nan"), float("nan")
    c.o_pad = c.w_pad = 0
    _, gw, _ = c.backward(grad=grad)
    assert gw[4, 3] == float("inf") and bool(torch.isnan(gw[9, 5]))
    gw[4, 3] = 2
    gw[9, 5] = 1
    want = torch.zeros(12, 32, device="cuda")
    want[4], want[2], want[9] = 2, 2, 1
    assert torch.equal(gw, want)


def test_the_same_bits_each_time(env):
    torch = env[0]
    c = _Call(env, _ids(8, 60000, 900), 900, 136, "f32", "f32")
    first = c.backward()[1].clone()
    for _ in range(3):
        assert torch.equal(c.backward()[1], first)


def test_gradient_against_differences(env):
    # the sum of out * r, whose gradient is that of out = r; linear, so that a difference is exact but for roundings
    torch, pkg, tok = env
    rows, dim = 40, 24
    c = _Call(env, _ids(6, 150, rows), rows, dim, "f32", "f32", scale=1.5, seed=2)
    r, gw, _ = c.backward()
    w, out, _ = c.forward()
    rng = np.random.default_rng(1)
    for v, j in zip(rng.integers(0, rows, 12), rng.integers(0, dim, 12)):
        ends = []
        for step in (-0.5, 0.5):
            w2 = w.clone()
            w2[v, j] += step
            _, out2, _ = c.forward(d_weight=w2.data_ptr())
            torch.cuda.synchronize()
            ends.append(float((out2.double() * r.double()).sum()))
        size = float((out.double() * r.double()).abs().sum())
        assert abs(ends[1] - ends[0] - float(gw[v, j])) <= size * 2.0**-22 + abs(float(gw[v, j])) * 2.0**-18


def test_streams_and_graphs(env):
    torch, pkg, tok = env
    c = _Call(env, _ids(9, 9000, 700), 700, 64, "bf16", "bf16")
    want = c.backward()[1].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = c.backward()[1]
    side.synchronize()
    assert torch.equal(got, want)
    # two graphs with a buffer each, replayed at once
    size = tok.embed_work_bytes(c.n, c.rows, c.dim)
    works = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    graphs, outs = [], []
    grad = c.backward()[0]
    for w in works:
        into = _array(torch, "bf16", c.rows, c.dim, 0, 0, fill=3.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.backward(work=w, grad=grad, into=into)
        outs.append(into[0])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_a_buffer_serves_fewer_ids(env):
    torch, pkg, tok = env
    for rows, dim in ((700, 8), (100257, 2048), (1 << 20, 256), (5000, 1031)):
        sizes = [tok.embed_work_bytes(n, rows, dim) for n in
                 (0, 1, 31, 32, 4095, 4096, 4097, 6144, 8192, 16384, 32767, 32768, 32769, 65536, 65537, 262143, 311296, 311297, 1 << 20,
                  1 << 22)]
        assert sizes == sorted(sizes)
        steps = [tok.embed_work_bytes(n, rows, dim) for n in range(0, 400000, 997)]
        assert steps == sorted(steps)
    big = tok.embed_work_bytes(40000, 300, 2048)
    work = torch.full((big,), 0xee, dtype=torch.uint8, device="cuda")
    for n in (1, 4096, 4097, 32768, 40000):
        c = _Call(env, _ids(n, n, 300), 300, 2048, "bf16", "bf16")
        grad, gw, _ = c.backward(work=work, work_bytes=big)
        assert torch.equal(gw, c.backward(grad=grad)[1])


def test_refusals(env):
    torch, pkg, tok = env
    c = _Call(env, _ids(1, 10, 20), 20, 8, "f32", "f32")
    for other in (dict(d_ids=None), dict(d_weight=None), dict(d_out=None), dict(weight_dtype=3), dict(out_dtype=-1), dict(dim=0),
                  dict(n_rows=0), dict(n_rows=(1 << 20) + 1), dict(n=1 << 31), dict(weight_stride=7), dict(out_stride=7),
                  dict(d_weight=c.d_ids.data_ptr() + 2), dict(d_ids=c.d_ids.data_ptr() + 1), dict(d_n=c.d_ids.data_ptr() + 4),
                  dict(dim=(1 << 20) + 1, weight_stride=1 << 21, out_stride=1 << 21)):
        with pytest.raises(pkg.TokError) as e:
            c.forward(**other)
        assert e.value.code == pkg.TOK_EINVAL, other
    for other in (dict(d_ids=None), dict(d_grad_out=None), dict(d_grad_weight=None), dict(d_work=None), dict(work_bytes=1),
                  dict(grad_out_dtype=7), dict(grad_weight_dtype=-1), dict(dim=0), dict(n_rows=0), dict(n=1 << 31),
                  dict(grad_out_stride=7), dict(grad_weight_stride=7), dict(d_grad_out=c.d_ids.data_ptr() + 1)):
        with pytest.raises(pkg.TokError) as e:
            c.backward(**other)
        assert e.value.code == pkg.TOK_EINVAL, other
    assert tok.embed_work_bytes(1 << 31, 20, 8) == 0 and tok.embed_work_bytes(5, 0, 8) == 0
    assert tok.embed_work_bytes(0, 1, 1) > 0
