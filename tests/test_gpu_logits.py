"""tok_logits_process, tok_logits_backward and tok_seen_bits against plain
implementations in 64 bits (numpy), and the gradient against differences of
the 64-bit forward formula.

Bounds.  With u = 2^-24, a score goes through at most six roundings of terms
that add up to S = (|x| max(1, r, 1/r) + f c + p + sum |bias|) / T, and the
temperature's reciprocal and product are two more: |error of y| <= 10 u S (+
the output type's unit roundoff times |y|, and half its smallest subnormal).  lse: the largest error of a y,
a relative error of at most 21 * 2^-22 for the exponentials that carry weight
(2^-22 each for ex2, and d log2(e) is rounded at |d| of up to about 20), (V /
128 + 40) u for a sum of V terms in threads and trees, and 2 u |lse|.
top is compared exactly, with the scores in 32-bit numpy."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"f32": (2.0 ** -24, 2.0 ** -149), "f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -133)}


@pytest.fixture(scope="module")
def env():
    import torch

    from exact_bpe_tokenization_utf_gb300 import _build
    _build.build()
    import exact_bpe_tokenization_utf_gb300 as pkg
    tok = pkg.Tokenizer.from_merges([], pkg.PATTERN_GPT2)
    yield torch, pkg, tok
    tok.close()


class _Case:
    """One call's inputs, on the host in full and on the device as the library takes them."""

    def __init__(self, torch, rows, V, kind="f32", seed=0, gen=0, bias=0, mask=None, seen=False, strengths=True,
                 pad=0, shift=0, share=False, logits=None, mask_rows=None):
        rng = np.random.default_rng(seed)
        self.torch, self.rows, self.V, self.kind = torch, rows, V, kind
        self.type = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]
        W = self.W = -(-V // 32)
        x = rng.normal(0, 3, (rows, V)).astype(np.float32) if logits is None else np.asarray(logits, np.float32)
        store = torch.zeros(shift + rows * (V + pad), dtype=self.type, device="cuda")
        view = store[shift:].view(rows, V + pad)
        view[:, :V] = torch.from_numpy(x).cuda().to(self.type)
        self.d = {"logits": view}
        self.stride = V + pad
        self.x = view[:, :V].float().cpu().numpy()
        one = np.ones(rows, np.float32)
        self.rep = (one + rng.random(rows) * 0.7).astype(np.float32) if strengths else one.copy()
        self.freq = (rng.random(rows) * 0.4).astype(np.float32) if strengths else 0 * one
        self.pres = (rng.random(rows) * 0.6 - 0.1).astype(np.float32) if strengths else 0 * one
        self.temp = (0.3 + rng.random(rows) * 1.5).astype(np.float32) if strengths else one.copy()
        self.gen = [np.zeros(0, np.int64)] * rows
        if gen:
            if share:  # prefixes of one sequence
                ids = rng.integers(0, V, gen)
                lens = np.linspace(0, gen, rows).astype(int)
                starts = np.zeros(rows, np.int64)
            else:
                lens = rng.integers(0, gen + 1, rows)
                lens[0] = gen
                if rows > 1:
                    lens[1] = 0
                starts = np.concatenate([[0], np.cumsum(lens)])[:-1]
                ids = rng.integers(0, V, max(1, int(lens.sum())))
                ids[rng.random(len(ids)) < 0.4] = int(rng.integers(0, V))  # one id many times
                bad = rng.random(len(ids)) < 0.1
                ids[bad] = rng.choice([-1, V, V + 5, 2**31 - 1, -2**31], int(bad.sum()))
            self.gen = [ids[s:s + n] for s, n in zip(starts, lens)]
            self._put(gen=ids.astype(np.int32), gen_start=starts.astype(np.int64), gen_len=lens.astype(np.int32))
        self.bias = [(np.zeros(0, np.int64), np.zeros(0, np.float32))] * rows
        if bias:
            self.bias = []
            for b in range(rows):
                n = int(rng.integers(0, bias + 1)) if b else bias
                ids = rng.integers(0, V, n)
                ids[rng.random(n) < 0.3] = int(rng.integers(0, V))  # the same id several times
                ids[rng.random(n) < 0.1] = rng.choice([-1, V, 2**31 - 1])
                self.bias.append((ids, rng.normal(0, 2, n).astype(np.float32)))
            off = np.concatenate([[0], np.cumsum([len(i) for i, _ in self.bias])])
            self._put(bias_off=off.astype(np.int64), bias_id=np.concatenate([i for i, _ in self.bias]).astype(np.int32),
                      bias=np.concatenate([v for _, v in self.bias]))
        bits = lambda p: rng.random((rows, W * 32)) < p  # noqa: E731
        words = lambda b: np.packbits(b, axis=1, bitorder="little").view(np.int32)  # noqa: E731
        self.seen = np.zeros((rows, V), bool)
        if seen:
            b = bits(0.2)
            self.seen = b[:, :V]
            self._put(seen=words(b))
        self.ok = np.ones((rows, V), bool)
        if mask is not None:
            b = bits(1.0)
            for k in range(rows):
                p = mask[k % len(mask)]
                b[k] = rng.random(W * 32) < p if p != "one" else False
                if p == "one":
                    b[k, int(rng.integers(0, V))] = True
            self._put(mask=words(b))
            if mask_rows is None:
                self.ok = b[:, :V]
            else:
                self._put(mask_row=np.asarray(mask_rows, np.int32))
                self.ok = np.stack([np.zeros(V, bool) if m == -1 else np.ones(V, bool) if m < 0 else b[m, :V] for m in mask_rows])
        self.pick = rng.integers(0, V, rows).astype(np.int32)
        if rows > 2:
            self.pick[2] = -1
        if strengths:
            self._put(repetition=self.rep, frequency=self.freq, presence=self.pres, temperature=self.temp)
        self._put(pick=self.pick)

    def _put(self, **arrays):
        for k, v in arrays.items():
            self.d[k] = self.torch.from_numpy(np.ascontiguousarray(v)).cuda()

    def p(self, k):
        return self.d[k].data_ptr() if k in self.d else None

    def args(self, pkg, out=True, out_pad=0, stats=True, **other):
        t = self.torch
        if out:
            self.d["out"] = t.full((self.rows, self.V + out_pad), 7.0, dtype=self.type, device="cuda")
        if stats:
            self.d["top"] = t.full((self.rows,), -9, dtype=t.int32, device="cuda")
            self.d["lse"], self.d["logprob"] = (t.full((self.rows,), 777.0, device="cuda") for _ in range(2))
        f = dict(d_logits=self.p("logits"), logits_stride=self.stride, d_out=self.p("out") if out else None,
                 out_stride=self.V + out_pad, dtype={"f32": 0, "f16": 1, "bf16": 2}[self.kind], rows=self.rows, n_logits=self.V,
                 d_seen=self.p("seen"), seen_stride=self.W, d_gen=self.p("gen"), d_gen_start=self.p("gen_start"),
                 d_gen_len=self.p("gen_len"), d_repetition=self.p("repetition"), d_frequency=self.p("frequency"),
                 d_presence=self.p("presence"), d_temperature=self.p("temperature"), d_bias_off=self.p("bias_off"),
                 d_bias_id=self.p("bias_id"), d_bias=self.p("bias"), d_mask=self.p("mask"), mask_stride=self.W,
                 d_mask_row=self.p("mask_row"), d_pick=self.p("pick"), d_top=self.p("top"), d_lse=self.p("lse"),
                 d_logprob=self.p("logprob"))
        f.update(other)
        return pkg.LogitsArgs(**f)

    def row(self, b, dtype=np.float64):
        """(scores before the temperature, factor of the repetition penalty, S) of row b by the definition."""
        V, one = self.V, dtype(1)
        x = self.x[b].astype(dtype)
        ids = self.gen[b][(self.gen[b] >= 0) & (self.gen[b] < V)]
        c = np.bincount(ids, minlength=V).astype(dtype)
        r = dtype(self.rep[b])
        hit = (c > 0) | self.seen[b]
        with np.errstate(all="ignore"):
            factor = np.where(hit, np.where(x > 0, one / r, r), one)
            z = np.where(hit, np.where(x > 0, x / r, x * r), x)
            z = np.where(c > 0, z - dtype(self.freq[b]) * c - dtype(self.pres[b]), z)
            total, size = np.zeros(V, dtype), np.zeros(V)
            has = np.zeros(V, bool)
            for i, v in zip(*self.bias[b]):
                if 0 <= i < V:
                    total[i] = dtype(v) if not has[i] else total[i] + dtype(v)
                    has[i] = True
                    size[i] += abs(float(v))
            z = np.where(has, z + total, z)
            S = np.abs(x.astype(np.float64)) * max(float(r), 1 / float(r), 1) + float(self.freq[b]) * c + abs(float(self.pres[b])) + size
        return np.where(self.ok[b], z, dtype(-np.inf)), factor, S

    def check(self, out=True, stats=True, out_pad=0):
        host = {k: self.d[k].float().cpu().numpy() if k != "top" else self.d[k].cpu().numpy()
                for k in (("out",) if out else ()) + (("top", "lse", "logprob") if stats else ())}
        unit, tiny = ROUND[self.kind]
        for b in range(self.rows):
            z, _, S = self.row(b)
            T = float(self.temp[b])
            y, E = z / T, 10 * U * S / T
            fine = np.isfinite(y)
            if out:
                got = host["out"][b, :self.V].astype(np.float64)
                assert (host["out"][b, self.V:] == 7.0).all()
                assert np.array_equal(got[~fine], y[~fine], equal_nan=True)
                err = np.abs(got[fine] - y[fine])
                assert (err <= E[fine] + (unit + U) * np.abs(y[fine]) + tiny).all(), (b, err.max())
            if not stats:
                continue
            z32 = self.row(b, np.float32)[0]
            pick = int(self.pick[b])
            if np.isnan(y).any():
                assert host["top"][b] == -1 and np.isnan(host["lse"][b]) and np.isnan(host["logprob"][b])
                continue
            top = int(np.argmax(z32)) if z32.max() > -np.inf else -1
            assert host["top"][b] == top, b
            if top < 0:
                assert host["lse"][b] == -np.inf and host["logprob"][b] == -np.inf
                continue
            m = y.max()
            if m == np.inf:
                assert host["lse"][b] == np.inf
                continue
            lse = m + math.log(np.exp(y - m).sum())
            tol = E[fine].max() + 21 * 2.0 ** -22 + (self.V / 128 + 40) * U + 2 * U * abs(lse)
            assert abs(host["lse"][b] - lse) <= tol, (b, host["lse"][b], lse)
            at = pick if pick >= 0 else top
            if at >= self.V or y[at] == -np.inf:
                assert host["logprob"][b] == -np.inf
            else:
                assert abs(host["logprob"][b] - (y[at] - lse)) <= 2 * tol + E[at] + 2 * U * (abs(y[at]) + abs(lse)), b


def _run(env, c, sync=True, out=True, **other):
    torch, pkg, tok = env
    tok.process_logits_device(c.args(pkg, out=out, **other), torch.cuda.current_stream().cuda_stream)
    return c


SIZES = [1, 2, 7, 31, 32, 33, 63, 257, 1000, 4095, 4096, 4097, 8200, 16385]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_everything_on(env, V, kind):
    torch = env[0]
    for seed, (rows, pad, shift, out_pad) in enumerate([(1, 0, 0, 0), (3, 0, 0, 0), (4, 1, 3, 0), (5, -V % 8, 0, -V % 8), (3, 5, 1, 2)]):
        c = _Case(torch, rows, V, kind, seed, gen=40, bias=9, mask=[0.9, 1.0, 0.03, "one"], seen=True, pad=pad, shift=shift)
        _run(env, c, out_pad=out_pad).check(out_pad=out_pad)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("what", ["nothing", "gen", "bias", "mask", "seen", "strengths"])
def test_one_rule_at_a_time(env, what, kind):
    torch = env[0]
    rules = dict(gen=dict(gen=300), bias=dict(bias=40), mask=dict(mask=[0.5, 0.999]), seen=dict(seen=True)).get(what, {})
    for rows, V in ((2, 50257), (3, 9001)):
        c = _Case(torch, rows, V, kind, 3, strengths=what in ("strengths", "gen", "seen"), **rules)
        _run(env, c).check()
        _run(env, c, out=False).check(out=False)
        # without the results that are optional
        args = c.args(env[1], stats=False, d_top=None, d_lse=None, d_logprob=None)
        env[2].process_logits_device(args)
        c.check(stats=False)


@pytest.mark.parametrize("rows", [1, 2, 9, 40, 160, 700])
def test_rows(env, rows):
    torch = env[0]
    c = _Case(torch, rows, 12_345, "bf16", rows, gen=200, bias=20, mask=[1.0, 0.9, 0.01], seen=True, pad=7)
    _run(env, c).check()
    _run(env, c, out=False).check(out=False)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_widest_rows(env, kind):
    c = _Case(env[0], 2, 1 << 20, kind, 1, gen=5000, bias=100, mask=[0.7, 0.001], seen=True)
    _run(env, c).check()
    c = _Case(env[0], 3, (1 << 20) - 3, kind, 1, gen=70_000, seen=True)
    _run(env, c).check()


def test_long_and_shared_histories(env):
    torch = env[0]
    c = _Case(torch, 33, 1500, "f32", 1, gen=20_000, share=True, mask=[0.9])
    _run(env, c).check()
    c = _Case(torch, 2, 40_000, "f16", 2, gen=90_000, bias=2000)
    _run(env, c).check()
    # an id more often than 16 bits count
    c = _Case(torch, 1, 50, "f32", 3, gen=10)
    c.gen = [np.full(70_001, 33)]
    c.freq[:] = 2.0 ** -12
    c._put(gen=c.gen[0].astype(np.int32), gen_len=np.array([70_001], np.int32), frequency=c.freq)
    _run(env, c).check()
    # a negative length is none
    c._put(gen_len=np.array([-5], np.int32))
    c.gen = [np.zeros(0, np.int64)]
    _run(env, c).check()


def test_bias_over_the_whole_row(env):
    c = _Case(env[0], 2, 5000, "f32", 4, bias=12_000, mask=[0.8])
    _run(env, c).check()


@pytest.mark.parametrize("V", [50, 5000])
def test_biases_are_added_in_the_lists_order(env, V):
    # ((x + b1) + b2) + ... in 32 bits, bit for bit: large values of both signs on the same few tokens
    torch = env[0]
    c = _Case(torch, 3, V, "f32", 15, bias=120, strengths=False)
    rng = np.random.default_rng(15)
    for b in range(3):
        ids, vals = c.bias[b]
        few = rng.random(len(ids)) < 0.7
        ids[few] = rng.integers(0, 5, int(few.sum()))
        vals[:] = (vals * 2.0 ** rng.integers(0, 26, len(vals))).astype(np.float32)
    c.bias[0][0][:3], c.bias[0][1][:3] = [7, 7, 7], [2.0 ** 24, -2.0 ** 24, 3.0]
    c.d["logits"][0, 7] = c.x[0, 7] = 1.0
    want = c.x.copy()
    for b in range(3):
        for i, v in zip(*c.bias[b]):
            if 0 <= i < V:
                want[b, i] += v
    c._put(bias_id=np.concatenate([i for i, _ in c.bias]).astype(np.int32), bias=np.concatenate([v for _, v in c.bias]))
    _run(env, c)
    assert np.array_equal(c.d["out"].cpu().numpy(), want)
    assert c.d["top"].cpu().tolist() == want.argmax(1).tolist()


def test_masked_places_are_not_looked_at(env):
    torch = env[0]
    for kind in ("f32", "f16", "bf16"):
        for V in (40, 20_003):
            c = _Case(torch, 6, V, kind, 5, gen=30, bias=5, mask=[0.5, 0.0, "one", 0.95, 1.0, 0.1], seen=True)
            bad = torch.tensor([math.nan, math.inf, -math.inf], device="cuda").repeat(6 * V)[:6 * V].view(6, V).to(c.type)
            ok = torch.from_numpy(c.ok.copy()).cuda()
            c.d["logits"][:, :V] = torch.where(ok, c.d["logits"][:, :V], bad)
            c.x = c.d["logits"][:, :V].float().cpu().numpy()
            _run(env, c).check()
            _run(env, c, out=False).check(out=False)


@pytest.mark.parametrize("value", [-math.inf, math.inf, math.nan, -65504.0, -3.3895313892515355e38])
def test_special_logits(env, value):
    # in one place, and in the whole row (a mask of the type's lowest value among them)
    torch = env[0]
    for kind in ("f32", "bf16") if abs(value) > 1e5 and math.isfinite(value) else ("f32", "f16", "bf16"):
        for V in (5, 70, 9000):
            x = np.random.default_rng(1).normal(0, 1, (4, V)).astype(np.float32)
            x[0, V // 2] = value
            x[1] = value
            x[2] = value
            x[2, V - 1] = 1.5
            c = _Case(torch, 4, V, kind, 6, logits=x, strengths=False, gen=1)
            c.pick[:] = V - 1
            c._put(pick=c.pick)
            _run(env, c).check()
            _run(env, c, out=False).check(out=False)


@pytest.mark.parametrize("temp", [1.0, 1e-9, 1e-3])
@pytest.mark.parametrize("value", [-1e35, -1e30, -1e15, -1e10, -3e9, -7e8, -4e8, 4e8, 7e8, 3e9, 1e10, 1e20, 1.0])
def test_scores_far_from_0(env, value, temp):
    # rows of one large value (a mask that was added to the scores), of large ones that differ, and ordinary ones
    # over a small temperature.  The bounds are the module's, with the errors of those scores alone that carry weight
    # (within 60 of the largest: a row has fewer than 2^20 others)
    torch, pkg, tok = env
    for kind in ("f32", "bf16"):
        for V in (5, 70, 9000, 60_000):
            rng = np.random.default_rng(2)
            x = rng.normal(0, 1, (5, V)).astype(np.float32)
            x[0, V // 2] = value
            x[1] = value
            x[2] = value
            x[2, V - 1] = 1.5
            x[3] *= np.float32(value)
            c = _Case(torch, 5, V, kind, 6, logits=x, strengths=False)
            c.temp[:] = temp
            c.pick[:] = [V - 1, 0, 0, -1, -1]
            c._put(pick=c.pick, temperature=c.temp)
            _run(env, c)
            top, lse, logprob = (c.d[k].cpu().numpy() for k in ("top", "lse", "logprob"))
            for b in range(5):
                z, _, S = c.row(b)
                y, E = z / float(c.temp[b]), 10 * U * S / float(c.temp[b])
                assert top[b] == int(np.argmax(c.row(b, np.float32)[0]))
                m = y.max()
                want = m + math.log(np.exp(y - m).sum())
                tol = E[y >= m - 60].max() + 21 * 2.0 ** -22 + (V / 128 + 40) * U + 2 * U * abs(want)
                at = int(c.pick[b]) if c.pick[b] >= 0 else int(top[b])
                with np.errstate(all="ignore"):  # (what 32 bits do not hold is infinite)
                    y32, want32 = np.float32(y[at]), np.float32(want)
                if np.isinf(y32) or np.isinf(want32):
                    assert np.isfinite(want32) or lse[b] == want32, (kind, V, b)
                    assert logprob[b] == -np.inf if y32 < np.inf else np.isnan(logprob[b]), (kind, V, b)
                    continue
                assert abs(lse[b] - want) <= tol, (kind, V, b, lse[b], want)
                assert abs(logprob[b] - (y[at] - want)) <= 2 * tol + E[at] + 2 * U * (abs(y[at]) + abs(want)), (kind, V, b)


def test_ties_go_to_the_lowest_token(env):
    torch = env[0]
    for V in (100, 6001, 100_257):
        x = np.zeros((5, V), np.float32)
        x[1] = -2
        x[2, V // 3:] = 4
        x[3, [V - 1, V // 2]] = 9
        x[4, 0] = x[4, V - 1] = 1
        for kind in ("f32", "f16", "bf16"):
            c = _Case(torch, 5, V, kind, 7, logits=x, strengths=False)
            _run(env, c).check()
            assert c.d["top"].cpu().tolist() == [0, 0, V // 3, V // 2, 0]
    # a penalised score that rounds to another one's exact value
    x = np.full((1, 64), -1.0, np.float32)
    x[0, 7], x[0, 40], x[0, 50] = 12.0, 10.0, 12.0
    c = _Case(torch, 1, 64, "f32", 8, logits=x, strengths=False)
    c.rep[:] = 1.2
    c.seen[0, [7, 50]] = True
    w = np.zeros((1, 64), bool)
    w[0, [7, 50]] = True
    c._put(repetition=c.rep, seen=np.packbits(w, axis=1, bitorder="little").view(np.int32))
    _run(env, c).check()


def test_mask_rows(env):
    torch = env[0]
    for V in (33, 9000):
        c = _Case(torch, 6, V, "bf16", 9, mask=[0.9, 0.02, 1.0, "one"], mask_rows=[3, 0, -1, -2, 0, 1], gen=10)
        _run(env, c).check()


def test_picks_outside_the_row(env):
    torch = env[0]
    c = _Case(torch, 4, 1000, "f32", 10, mask=[0.5, 0.0])
    c.pick[:] = [1000, 5, -3, 2**31 - 1]
    c._put(pick=c.pick)
    _run(env, c).check()
    c = _Case(torch, 4, 1000, "f32", 10, mask=[0.5, 0.0])
    del c.d["pick"]
    c.pick[:] = -1
    _run(env, c).check()


def test_in_place_other_stream_and_graph(env):
    torch, pkg, tok = env
    c = _Case(torch, 3, 10_001, "f16", 11, gen=50, bias=10, mask=[0.9], seen=True, pad=3, shift=1)
    src = c.d["logits"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = c.args(pkg, out=False)
    args.d_out, args.out_stride = c.p("logits"), c.stride
    with torch.cuda.stream(s):
        tok.process_logits_device(args, s.cuda_stream)
    s.synchronize()
    c.d["out"] = c.d["logits"][:, :c.V].clone()
    c.check()
    c.d["logits"].copy_(src)
    args = c.args(pkg)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tok.process_logits_device(args, torch.cuda.current_stream().cuda_stream)
    c.d["logits"].copy_(src.flip(0))
    c.x = c.d["logits"][:, :c.V].float().cpu().numpy()
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_the_same_call_gives_the_same_bits(env):
    torch = env[0]
    c = _Case(torch, 5, 60_000, "f32", 12, gen=5000, bias=500, mask=[0.9], seen=True)
    got = []
    for _ in range(4):
        _run(env, c)
        got.append([c.d[k].clone() for k in ("out", "top", "lse", "logprob")])
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(got[0], g))


# --- gradient ----------------------------------------------------------------

def _grad_inputs(c, seed, dense=True, scalars=True):
    rng, t = np.random.default_rng(seed), c.torch
    go = t.from_numpy(rng.normal(0, 1, (c.rows, c.V)).astype(np.float32)).cuda().to(c.type)
    c.d["go"] = go
    c.go = go.double().cpu().numpy() if dense else np.zeros((c.rows, c.V))
    c.glse, c.glp = (rng.normal(0, 1, c.rows).astype(np.float32) * scalars for _ in range(2))
    c._put(glse=c.glse, glp=c.glp)


def _backward(env, c, dense=True, scalars=True, pad=0):
    torch, pkg, tok = env
    args = c.args(pkg, out=False)
    tok.process_logits_device(args)
    c.d["gx"] = torch.full((c.rows, c.V + pad), 7.0, dtype=c.type, device="cuda")
    if "bias" in c.d:
        c.d["gb"] = torch.full_like(c.d["bias"], 7.0)
    ga = pkg.LogitsGradArgs(d_grad_out=c.p("go") if dense else None, grad_out_stride=c.V, d_grad_lse=c.p("glse") if scalars else None,
                            d_grad_logprob=c.p("glp") if scalars else None, d_grad_logits=c.p("gx"), grad_logits_stride=c.V + pad,
                            d_grad_bias=c.p("gb"))
    tok.process_logits_backward_device(args, ga)


def _check_grad(c):
    """Against the formula in 64 bits, with the lse that the forward pass wrote.  The bound: exp(y - lse) is off by the
    error of y (10 u S), of lse's use (2 u |lse|), of d log2(e) (2 u 1.5 |d|) and of ex2 (2^-22), relatively; the sum of
    three terms, the two products and the factor are six more roundings, then the type's own."""
    unit, tiny = ROUND[c.kind]
    gx, lse = c.d["gx"].float().cpu().numpy(), c.d["lse"].cpu().numpy().astype(np.float64)
    top = c.d["top"].cpu().numpy()
    gb = c.d["gb"].cpu().numpy() if "bias" in c.d else None
    at = 0
    for b in range(c.rows):
        z, factor, S = c.row(b)
        T, glp = float(c.temp[b]), float(c.glp[b])
        cp = float(c.glse[b]) - glp if lse[b] > -np.inf else 0.0
        with np.errstate(all="ignore"):
            y = z / T
            d = np.where(np.isfinite(y), y - lse[b], 0.0)
            p = np.where(y > -np.inf, np.exp(d), 0.0) if cp else np.zeros(c.V)
        hit = np.zeros(c.V)
        pick = int(c.pick[b]) if c.pick[b] >= 0 else int(top[b])
        if 0 <= pick < c.V:
            hit[pick] = glp
        terms = np.abs(c.go[b]) + np.abs(cp) * p + np.abs(hit)
        dz = np.where(c.ok[b], (c.go[b] + cp * p + hit) / T, 0.0)
        rel = 10 * U * S / T + 2 * U * abs(lse[b] if cp else 0) + 3 * U * np.abs(d) + 2.0 ** -22
        rel[p == 0] = 0.0  # (a score of -inf has no error)
        err = np.where(c.ok[b], (np.abs(cp) * p * rel + 6 * U * terms) / T, 0.0)
        got = gx[b, :c.V].astype(np.float64)
        assert (gx[b, c.V:] == 7.0).all()
        want = dz * factor
        assert (np.abs(got - want) <= err * factor + unit * np.abs(want) * 1.01 + tiny + 2.0 ** -126).all(), \
            (b, np.abs(got - want).max())
        if gb is not None:
            for i, v in enumerate(c.bias[b][0]):
                w, e = (dz[v], err[v]) if 0 <= v < c.V else (0.0, 0.0)
                assert abs(gb[at + i] - w) <= e + 2 * U * abs(w) + 2.0 ** -126, (b, i)
            at += len(c.bias[b][0])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_gradient(env, V, kind):
    torch = env[0]
    for seed, (rows, pad, shift, gpad) in enumerate([(1, 0, 0, 0), (4, 0, 0, 0), (5, 1, 3, 0), (4, -V % 8, 0, -V % 8), (3, 5, 1, 2)]):
        c = _Case(torch, rows, V, kind, seed, gen=40, bias=9, mask=[0.9, 1.0, 0.03, 0.0, "one"], seen=True, pad=pad, shift=shift)
        for dense, scalars in ((True, True), (False, True), (True, False)):
            _grad_inputs(c, seed, dense, scalars)
            _backward(env, c, dense, scalars, gpad)
            _check_grad(c)


def test_gradient_rows_and_histories(env):
    torch = env[0]
    for c in (_Case(torch, 300, 20_011, "bf16", 1, gen=299, share=True, mask=[0.9, 0.01], seen=True, pad=5),
              _Case(torch, 2, 100_257, "f32", 2, gen=40_000, bias=300, seen=True),
              _Case(torch, 3, 5000, "f16", 3, bias=9000, mask=[0.8])):
        _grad_inputs(c, 4, dense=False)
        _backward(env, c, dense=False)
        _check_grad(c)


def test_gradient_ignores_what_the_mask_hides(env):
    torch = env[0]
    c = _Case(torch, 4, 3001, "f32", 5, mask=[0.5, 0.0, 0.9, "one"], gen=20)
    hidden = torch.from_numpy(~c.ok).cuda()
    c.d["logits"][:, :c.V][hidden] = math.nan
    c.x = c.d["logits"][:, :c.V].float().cpu().numpy()
    _grad_inputs(c, 6)
    c.d["go"][hidden] = math.nan
    c.go = np.where(c.ok, c.go, 0.0)
    _backward(env, c)
    _check_grad(c)
    # a row whose scores are all -inf: nothing through lse
    c = _Case(torch, 2, 50, "f32", 6, logits=np.full((2, 50), -np.inf), strengths=False)
    _grad_inputs(c, 7)
    _backward(env, c)
    _check_grad(c)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [33, 1000, 50_257])
def test_gradient_of_negative_picks_without_a_top(env, V, kind):
    # padded rows: a pick of -1 and no d_top, so that no token is the row's pick
    torch, pkg, tok = env
    for dense in (True, False):
        c = _Case(torch, 5, V, kind, 13, gen=20, mask=[0.9, 1.0], seen=True)
        c.pick[[0, 1, 3]] = [-1, -1, -2**31]
        c._put(pick=c.pick)
        _grad_inputs(c, 14, dense)
        args = c.args(pkg, out=False)
        tok.process_logits_device(args)
        args.d_top = None
        c.d["gx"] = torch.full((c.rows, c.V), 7.0, dtype=c.type, device="cuda")
        tok.process_logits_backward_device(args, pkg.LogitsGradArgs(
            d_grad_out=c.p("go") if dense else None, grad_out_stride=V, d_grad_lse=c.p("glse"), d_grad_logprob=c.p("glp"),
            d_grad_logits=c.p("gx"), grad_logits_stride=V))
        c.d["top"].fill_(-1)
        _check_grad(c)


@pytest.mark.parametrize("temp", [1.1e-8, 1.3e-8, 1e30, 1e37])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_gradient_of_the_lowest_scores_at_any_temperature(env, kind, temp):
    # scores of -inf and of a type's lowest value next to a single 0: no NaN, whatever they are multiplied by
    torch = env[0]
    for V in (5, 40, 9001):
        x = np.full((2, V), -np.inf, np.float32)
        x[:, 1::3] = -3.38e38
        x[0, V // 2] = x[1, V - 1] = 0
        c = _Case(torch, 2, V, kind, 16, logits=x, strengths=False, gen=4)
        c.temp[:] = temp
        c._put(temperature=c.temp)
        for dense in (True, False):
            _grad_inputs(c, 17, dense)
            _backward(env, c, dense)
            _check_grad(c)


@pytest.mark.parametrize("value", [-1e35, -1e30, -1e15, -1e10, -3e9, -1e8, -2e7, 4e6, 1e8, 1e10, 1e20])
def test_gradient_of_scores_far_from_0(env, value):
    # At a temperature of 1 y is the logit itself.  exp(y - lse) is off by the roundings of the difference and of its
    # product with log2(e) (3 u |d|) and by ex2's 2^-22; it is at most 1 where lse, rounded, lies below the largest y.
    # The sum of the terms and its product are 6 roundings more, then the type's own.
    torch = env[0]
    for kind in ("f32", "bf16"):
        unit, tiny = ROUND[kind]
        for V in (5, 70, 9000, 60_000):
            rng = np.random.default_rng(2)
            x = rng.normal(0, 1, (4, V)).astype(np.float32)
            x[0] = value
            x[1, V // 2] = abs(value)
            x[2, 1:] = value
            x[3] *= np.float32(value)
            c = _Case(torch, 4, V, kind, 6, logits=x, strengths=False)
            for dense in (True, False):
                _grad_inputs(c, 18, dense)
                _backward(env, c, dense)
                gx, lse, top = (c.d[k].double().cpu().numpy() for k in ("gx", "lse", "top"))
                for b in range(4):
                    d = np.minimum(c.x[b].astype(np.float64) - lse[b], 0.0)
                    p, hit = np.exp(d), np.zeros(V)
                    hit[int(c.pick[b] if c.pick[b] >= 0 else top[b])] = float(c.glp[b])
                    cp = float(np.float32(c.glse[b]) - np.float32(c.glp[b]))
                    want = c.go[b] + cp * p + hit
                    size = np.abs(c.go[b]) + np.abs(cp) * p + np.abs(hit)
                    rel = 3 * U * np.abs(d) + 2.0 ** -22
                    if abs(lse[b]) < 2**20:
                        rel += 2 * U * (abs(lse[b]) + np.abs(c.x[b]))
                    err = np.abs(cp) * p * np.minimum(rel, 1.0) + 6 * U * size
                    assert (np.abs(gx[b] - want) <= err + unit * np.abs(want) * 1.01 + tiny + 2.0 ** -126).all(), (kind, V, b)


@pytest.mark.parametrize("temp", [1e-9, 1e-7])
def test_gradient_at_next_to_no_temperature(env, temp):
    # the largest score, and each one equal to it, has a weight of 1: lse is its y, rounded as exp's argument is
    torch, pkg, tok = env
    for kind in ("f32", "f16", "bf16"):
        for V in (33, 9000, 60_000):
            c = _Case(torch, 4, V, kind, 19, gen=20, bias=5, seen=True)
            c.temp[:] = temp
            c.rep[:] = 1.25 if temp < 1e-8 else 1.0
            c._put(temperature=c.temp, repetition=c.rep)
            _grad_inputs(c, 20, False)
            c._put(glp=0 * c.glp, glse=np.full(4, temp, np.float32))
            _backward(env, c, False)
            gx, top = c.d["gx"].double().cpu().numpy(), c.d["top"].cpu().numpy()
            for b in range(4):
                z32 = c.row(b, np.float32)[0]
                want = np.where(z32 == z32[top[b]], c.row(b)[1], 0.0)
                assert (np.abs(gx[b] - want) <= 2.0 ** -7 * want + 2.0 ** -24).all(), (kind, V, b)


def test_gradient_against_differences(env):
    # L = sum(grad_out * y) + grad_lse * lse + grad_logprob * logprob in 64 bits, central differences of step h:
    # the error is h^2 times a third derivative (at most about 10 / T^3) and 2^-52 |L| / h
    torch = env[0]
    rows, V, h = 2, 60, 1e-4
    c = _Case(torch, rows, V, "f32", 8, gen=25, bias=12, mask=[0.8, 1.0], seen=True)
    for b in range(rows):  # picks that the mask allows, logits away from the penalty's kink
        c.pick[b] = int(np.flatnonzero(c.ok[b])[b + 1])
    c._put(pick=c.pick)
    x = c.d["logits"][:, :V]
    x[x.abs() < 0.01] = 0.5
    c.x = x.float().cpu().numpy()
    _grad_inputs(c, 9)
    _backward(env, c)
    _check_grad(c)
    gx, gb = c.d["gx"].cpu().numpy(), c.d["gb"].cpu().numpy()
    base = c.x.astype(np.float64)

    def loss(b):
        y = c.row(b)[0] / float(c.temp[b])
        ok = c.ok[b]
        lse = np.log(np.exp(y[ok]).sum())
        return (c.go[b][ok] * y[ok]).sum() + c.glse[b] * lse + c.glp[b] * (y[c.pick[b]] - lse)

    at = 0
    for b in range(rows):
        scale = 10 / float(c.temp[b]) ** 3
        size = np.abs(c.go[b]).sum() * 20
        tol = scale * h * h * 10 + 2.0 ** -52 * size / h + 1e-5
        for v in range(V):
            c.x = base.copy()
            c.x[b, v] += h
            up = loss(b)
            c.x[b, v] -= 2 * h
            assert abs((up - loss(b)) / (2 * h) - gx[b, v]) <= tol, (b, v)
        c.x = base
        ids, vals = c.bias[b]
        for i in range(len(ids)):
            if not 0 <= ids[i] < V:
                assert gb[at + i] == 0
                continue
            keep = c.bias[b]
            d = []
            for s in (h, -h):
                w = vals.astype(np.float64).copy()
                w[i] += s
                c.bias[b] = (ids, w)
                d.append(loss(b))
            c.bias[b] = keep
            assert abs((d[0] - d[1]) / (2 * h) - gb[at + i]) <= tol, (b, i)
        at += len(ids)


@pytest.mark.parametrize("rows,kind", [(3, "bf16"), (200, "f32")])
def test_same_bits_each_time(env, rows, kind):
    torch, pkg, tok = env
    c = _Case(torch, rows, 50_001, kind, 12, gen=200, bias=30, mask=[0.9, 0.1, 1.0], seen=True, strengths=True)
    first = None
    for _ in range(20):
        _run(env, c)
        torch.cuda.synchronize()
        got = [c.d[k].clone().view(torch.int16 if k == "out" and kind != "f32" else torch.int32) for k in ("out", "top", "lse", "logprob")]
        assert first is None or all(torch.equal(g, f) for g, f in zip(got, first))
        first = first or got


@pytest.mark.parametrize("rows", [0, 1, 2])
def test_in_place_with_another_stride(env, rows):
    """Rows of out that begin inside other rows of the logits: refused; a single row has no stride."""
    torch, pkg, tok = env
    c = _Case(torch, 2, 100, "f32", 1)
    args = c.args(pkg, d_out=c.p("logits"), out_stride=101, logits_stride=100, rows=rows)
    if rows < 2:
        tok.process_logits_device(args)
    else:
        with pytest.raises(pkg.TokError) as e:
            tok.process_logits_device(args)
        assert e.value.code == pkg.TOK_EINVAL and "stride" in str(e.value)
        torch.cuda.synchronize()
        assert np.array_equal(c.d["logits"].cpu().numpy(), c.x)


@pytest.mark.parametrize("kind,by", [("f32", 1), ("f32", 2), ("f32", 3), ("f16", 1), ("bf16", 1)])
def test_scores_between_two_places_are_refused(env, kind, by):
    torch, pkg, tok = env
    c = _Case(torch, 3, 100, kind, 1)
    args = c.args(pkg)
    ga = dict(d_grad_out=c.p("logits"), grad_out_stride=100, d_grad_logits=c.p("out"), grad_logits_stride=100)
    calls = [lambda: tok.process_logits_device(c.args(pkg, d_logits=c.p("logits") + by)),
             lambda: tok.process_logits_device(c.args(pkg, d_out=c.p("out") + by))]
    for k in ("d_grad_out", "d_grad_logits"):
        calls.append(lambda k=k: tok.process_logits_backward_device(args, pkg.LogitsGradArgs(**{**ga, k: ga[k] + by})))
    for call in calls:
        with pytest.raises(pkg.TokError) as e:
            call()
        assert e.value.code == pkg.TOK_EINVAL and "multiple" in str(e.value)
    torch.cuda.synchronize()
    assert (c.d["out"] == 7.0).all()


def test_no_rows(env):
    # a batch of no rows as tensors have it: their addresses are NULL
    torch, pkg, tok = env
    f = torch.empty((0, 100), device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    shared = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert f.data_ptr() == none.data_ptr() == 0
    before = tok.launch_count
    args = pkg.LogitsArgs(d_logits=f.data_ptr(), logits_stride=100, d_out=f.data_ptr(), out_stride=100, rows=0, n_logits=100,
                          d_gen=shared.data_ptr(), d_gen_start=none.data_ptr(), d_gen_len=none.data_ptr(),
                          d_bias_off=off.data_ptr(), d_bias_id=none.data_ptr(), d_bias=f.data_ptr())
    tok.process_logits_device(args)
    tok.process_logits_backward_device(args, pkg.LogitsGradArgs(d_grad_logits=f.data_ptr(), grad_logits_stride=100))
    assert tok.launch_count == before


# --- refusals, seen bits -----------------------------------------------------

def test_refusals(env):
    torch, pkg, tok = env
    c = _Case(torch, 3, 100, "f32", 1, gen=5, bias=3, mask=[0.5], seen=True)
    for bad in (dict(d_logits=None), dict(dtype=3), dict(dtype=-1), dict(n_logits=0), dict(n_logits=(1 << 20) + 1),
                dict(logits_stride=99), dict(out_stride=99), dict(seen_stride=3), dict(mask_stride=3), dict(d_gen_len=None),
                dict(d_gen_start=None), dict(d_bias_id=None), dict(d_bias=None), dict(d_mask=None, d_mask_row=c.p("pick"))):
        args = c.args(pkg, **bad)
        for call in (lambda: tok.process_logits_device(args),
                     lambda: tok.process_logits_backward_device(args, pkg.LogitsGradArgs(d_grad_logits=c.p("out"), grad_logits_stride=100))):
            if "out_stride" in bad or "d_logits" in bad:
                args.d_out = c.p("out")
            with pytest.raises(pkg.TokError) as e:
                call()
            assert e.value.code == pkg.TOK_EINVAL and "logits" in str(e.value), bad
    args = c.args(pkg)
    for bad in (dict(), dict(d_grad_logits=c.p("out"), grad_logits_stride=99),
                dict(d_grad_logits=c.p("out"), grad_logits_stride=100, d_grad_out=c.p("out"), grad_out_stride=99)):
        with pytest.raises(pkg.TokError) as e:
            tok.process_logits_backward_device(args, pkg.LogitsGradArgs(**bad))
        assert e.value.code == pkg.TOK_EINVAL
    ok = dict(d_grad_logits=c.p("out"), grad_logits_stride=100, d_grad_logprob=c.p("lse"))
    for gone in (dict(d_lse=None), dict(d_pick=None, d_top=None)):
        with pytest.raises(pkg.TokError) as e:
            tok.process_logits_backward_device(c.args(pkg, **gone), pkg.LogitsGradArgs(**ok))
        assert e.value.code == pkg.TOK_EINVAL
    L = pkg.lib()
    assert L.tok_logits_process(None, args._addr, None) == pkg.TOK_EINVAL
    assert L.tok_logits_process(tok._h, None, None) == pkg.TOK_EINVAL
    assert L.tok_logits_backward(tok._h, args._addr, None, None) == pkg.TOK_EINVAL
    torch.cuda.synchronize()
    assert (c.d["out"] == 7.0).all() and (c.d["top"] == -9).all()
    tok.process_logits_device(c.args(pkg, rows=0))
    assert (c.d["top"] == -9).all()
    one = torch.zeros(8, dtype=torch.int64, device="cuda").data_ptr()
    good = [one, one, 1, 100, one, 4]
    for at, v in ((0, None), (1, None), (2, 0), (3, 0), (3, (1 << 20) + 1), (4, None), (5, 3)):
        bad = list(good)
        bad[at] = v
        with pytest.raises(pkg.TokError) as e:
            tok.seen_bits_device(*bad)
        assert e.value.code == pkg.TOK_EINVAL and "seen bits" in str(e.value)


@pytest.mark.parametrize("n_logits", [1, 31, 32, 33, 1257, 100_257, 1 << 20])
@pytest.mark.parametrize("n,most", [(1, 0), (1, 1), (1, 70_000), (2, 33), (5, 3000), (70, 500), (900, 40)])
def test_seen_bits(env, n_logits, n, most):
    torch, pkg, tok = env
    rng = np.random.default_rng(n + most)
    lens = rng.integers(0, most + 1, n)
    lens[-1] = most
    off = np.concatenate([[0], np.cumsum(lens)])
    ids = (rng.random(max(1, off[-1])) ** 4 * n_logits).astype(np.int64)
    bad = rng.random(len(ids)) < 0.1
    ids[bad] = rng.choice([-1, n_logits, 2**31 - 1, -2**31], int(bad.sum()))
    W = -(-n_logits // 32)
    before = rng.integers(-2**31, 2**31, (n, W)).astype(np.int32) & rng.integers(-2**31, 2**31, (n, W)).astype(np.int32)
    want = np.zeros((n, W), np.uint32)
    for k in range(n):
        part = ids[off[k]:off[k + 1]]
        part = np.unique(part[(part >= 0) & (part < n_logits)])
        np.bitwise_or.at(want[k], part >> 5, np.uint32(1) << (part & 31).astype(np.uint32))
    d_ids, d_off = torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(off.astype(np.int64)).cuda()
    for keep in (False, True):
        d = torch.full((n, W + 2), -9, dtype=torch.int32, device="cuda")
        d[:, :W] = torch.from_numpy(before).cuda()
        tok.seen_bits_device(d_ids.data_ptr(), d_off.data_ptr(), n, n_logits, d.data_ptr(), W + 2, keep,
                             torch.cuda.current_stream().cuda_stream)
        got = d.cpu().numpy()
        assert (got[:, W:] == -9).all()
        assert np.array_equal(got[:, :W].view(np.uint32), want | (before.view(np.uint32) if keep else 0)), keep
