"""A batch decodes under a grammar, from texts to texts: encode, places in a
paged cache, the prompts' token sets, and then per token the grammar's masks,
the rules on the scores, the choice, the next place, and the blocks of finished
requests back; at the end the gradient of the choices' log-probabilities.

The language model is a stand-in with random weights: a request's hidden row is
its last token's embedding plus the mean of what its cache holds.  It is there
so that every operator reads and writes what it would next to a real one.

    python examples/constrained_decode.py
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import exact_bpe_tokenization_utf_gb300 as bpe  # noqa: E402


def record_grammar(name_len=12, digits=4):
    """The byte automaton of {"name": "<lower-case words>", "count": <digits>}."""
    nxt, accept = [], []

    def state(final=False):
        nxt.append([-1] * 256)
        accept.append(final)
        return len(nxt) - 1

    def literal(s, text):
        for c in text:
            if nxt[s][c] < 0:
                nxt[s][c] = state()
            s = nxt[s][c]
        return s

    s = literal(state(), b'{"name": "')
    ends = []
    for k in range(name_len):
        t = state()
        for c in b"abcdefghijklmnopqrstuvwxyz" + (b" " if k else b""):
            nxt[s][c] = t
        s = t
        ends.append(s)
    quote = state()
    for e in ends:
        nxt[e][ord('"')] = quote
    s = literal(quote, b', "count": ')
    last = []
    for _ in range(digits):
        t = state()
        for c in b"0123456789":
            nxt[s][c] = t
        s = t
        last.append(s)
    closed = state(True)
    for e in last:
        nxt[e][ord("}")] = closed
    return np.array(nxt, np.int32), np.array(accept, np.uint8)


class Decoder:
    """The buffers of a batch of requests and the calls of a step."""

    def __init__(self, tok, prompts, nxt, accept, max_new=48, block=16, width=64, seed=1):
        self.tok, self.n, self.block, self.max_new = tok, len(prompts), block, max_new
        self.V, self.eos = tok.n_vocab + 1, tok.n_vocab
        self.words = -(-self.V // 32)
        self.grammar = bpe.Grammar(tok, nxt, accept)
        self.stream = torch.cuda.current_stream().cuda_stream
        n = self.n

        def dev(a, dtype):
            return torch.as_tensor(np.asarray(a), dtype=dtype, device="cuda")

        def zeros(shape, dtype):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        # texts to ids
        text = b"".join(prompts)
        starts = np.concatenate([[0], np.cumsum([len(p) for p in prompts])])
        self.cap = max(1, len(text))
        d_text = dev(np.frombuffer(text + b"\0", np.uint8).copy(), torch.uint8)
        d_starts = dev(starts, torch.int64)
        self.ids = zeros(self.cap, torch.int32)
        self.item_off = zeros(n + 1, torch.int64)
        self.status = zeros(4, torch.int64)
        tok.encode_batch_device(d_text.data_ptr(), len(text), d_starts.data_ptr(), n, self.ids.data_ptr(), self.cap,
                                self.item_off.data_ptr(), self.status.data_ptr(), self.stream)
        if int(self.status[0]) != bpe.TOK_OK:
            raise bpe.TokError(int(self.status[0]), "a prompt could not be encoded")

        # the paged cache, with exactly the blocks that the longest outcome takes
        longest = int((self.item_off[1:] - self.item_off[:-1]).max()) + max_new
        self.max_blocks = -(-longest // block)
        self.n_blocks = n * self.max_blocks
        self.table = zeros((n, self.max_blocks), torch.int32)
        self.free = torch.arange(self.n_blocks, dtype=torch.int32, device="cuda")
        self.n_free = dev([self.n_blocks], torch.int64)
        self.seq_len = zeros(n, torch.int64)
        self.slot = zeros(max(self.cap, n), torch.int64)
        self.pos = zeros(max(self.cap, n), torch.int32)
        self.req = zeros(max(self.cap, n), torch.int32)
        self.released = zeros(n, torch.uint8)

        # the model
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn(self.V, width, generator=g, device="cuda")
        self.head = (torch.randn(self.V, width, generator=g, device="cuda") / width ** 0.5).bfloat16()
        self.cache = zeros((self.n_blocks * block, width), torch.float32)
        self.last = torch.zeros(n, width, device="cuda")

        # the rules on the scores
        self.seen = zeros((n, self.words), torch.int32)
        self.mask = zeros((n, self.words), torch.int32)
        self.states = [zeros(n, torch.int32), zeros(n, torch.int32)]
        self.gen = torch.full((n, max_new), -1, dtype=torch.int32, device="cuda")
        self.gen_start = dev(np.arange(n) * max_new, torch.int64)
        self.gen_len = zeros(n, torch.int32)
        self.repetition = torch.full((n,), 1.3, device="cuda")
        self.frequency = torch.full((n,), 0.4, device="cuda")
        self.presence = torch.full((n,), 0.2, device="cuda")
        self.temperature = torch.full((n,), 0.8, device="cuda")
        # the end token is liked a little more than the model says
        self.bias_off = dev(np.arange(n + 1), torch.int64)
        self.bias_id = dev([self.eos] * n, torch.int32)
        self.bias = dev([1.5] * n, torch.float32)
        self.logits = zeros((n, self.V), torch.bfloat16)
        self.top = zeros(n, torch.int32)
        self.lse = zeros(n, torch.float32)
        self.logprob = zeros(n, torch.float32)
        self.score = torch.zeros(n, device="cuda")
        self.args = bpe.LogitsArgs(
            d_logits=self.logits.data_ptr(), logits_stride=self.V, dtype=bpe.DTYPE_BF16, rows=n, n_logits=self.V,
            d_seen=self.seen.data_ptr(), seen_stride=self.words, d_gen=self.gen.data_ptr(),
            d_gen_start=self.gen_start.data_ptr(), d_gen_len=self.gen_len.data_ptr(),
            d_repetition=self.repetition.data_ptr(), d_frequency=self.frequency.data_ptr(),
            d_presence=self.presence.data_ptr(), d_temperature=self.temperature.data_ptr(),
            d_bias_off=self.bias_off.data_ptr(), d_bias_id=self.bias_id.data_ptr(), d_bias=self.bias.data_ptr(),
            d_mask=self.mask.data_ptr(), mask_stride=self.words, d_top=self.top.data_ptr(), d_lse=self.lse.data_ptr(),
            d_logprob=self.logprob.data_ptr())

        # the prompts go into the cache, and their token sets to the penalty
        tok.seen_bits_device(self.ids.data_ptr(), self.item_off.data_ptr(), n, self.V, self.seen.data_ptr(), self.words,
                             stream=self.stream)
        self._append(self.ids, self.item_off, self.cap)

    def _append(self, ids, item_off, cap):
        """Tokens item_off[k] .. item_off[k + 1] of ids into request k's cache."""
        args = bpe.PagedArgs(
            d_item_off=item_off.data_ptr(), d_ctx_len=self.seq_len.data_ptr(), n=self.n, block_size=self.block,
            d_table=self.table.data_ptr(), table_stride=self.max_blocks, max_blocks=self.max_blocks,
            d_free=self.free.data_ptr(), d_n_free=self.n_free.data_ptr(), d_n_free_out=self.n_free.data_ptr(),
            d_slot=self.slot.data_ptr(), d_pos=self.pos.data_ptr(), d_req=self.req.data_ptr(), cap=cap,
            d_seq_len=self.seq_len.data_ptr(), d_status=self.status.data_ptr())
        self.tok.paged_assign_device(args, self.stream)
        at = self.slot[:cap] >= 0   # (a padded batch: the rest is -1)
        row = self.embed[ids[:cap].clamp(min=0).long()]
        self.cache[self.slot[:cap][at]] = row[at]
        self.last.index_copy_(0, self.req[:cap][at].long(), row[at])  # (the stand-in keeps one of a request's rows)

    def _model(self):
        """The stand-in: what a request's blocks hold, averaged, and its last row."""
        longest = self.max_blocks * self.block
        at = torch.arange(longest, device="cuda")
        slots = self.table.long()[:, at // self.block] * self.block + at % self.block
        there = (at[None, :] < self.seq_len[:, None]).float()
        mean = (self.cache[slots] * there[..., None]).sum(1) / self.seq_len.clamp(min=1)[:, None].float()
        return (self.last + mean).bfloat16()

    def step(self):
        """One token for every request that has not ended; False once all have."""
        n, s = self.n, self.stream
        self.hidden = self._model()
        torch.mm(self.hidden, self.head.t(), out=self.logits)
        self.tok.process_logits_device(self.args, s)
        chosen = self.top.clone()                      # -1: the grammar leaves nothing, the request has ended
        alive = (chosen >= 0) & (chosen != self.eos)
        self.score += torch.where(chosen >= 0, self.logprob, torch.zeros_like(self.logprob))
        # the next masks, from the states after the chosen tokens
        before, after = self.states
        self.grammar.mask_device(before.data_ptr(), chosen.data_ptr(), None, n, self.eos, after.data_ptr(), self.V,
                                 self.mask.data_ptr(), self.words, s)
        self.states = [after, before]
        # the chosen tokens into the cache: one or none each
        step_off = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
        step_off[1:] = alive.long().cumsum(0)
        ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        ids[:int(step_off[n])] = chosen[alive]
        self._append(ids, step_off, n)
        at = self.gen_len.long().clamp(max=self.max_new - 1)[:, None]
        self.gen.scatter_(1, at, torch.where(alive, chosen, self.gen.gather(1, at)[:, 0])[:, None])
        self.gen_len += alive.int()
        # what has ended gives its blocks back, once
        self.release((~alive).byte())
        return bool(alive.any())

    def release(self, done):
        done = done * (1 - self.released)
        self.tok.paged_release_device(self.seq_len.data_ptr(), done.data_ptr(), self.n, self.block, self.table.data_ptr(),
                                      self.max_blocks, self.max_blocks, self.free.data_ptr(), self.n_blocks,
                                      self.n_free.data_ptr(), self.n_free.data_ptr(), self.status.data_ptr(), self.stream)
        self.released |= done
        self.seq_len *= (1 - done.long())

    def run(self):
        n = self.n
        before, after = self.states
        self.grammar.mask_device(before.data_ptr(), None, None, n, self.eos, after.data_ptr(), self.V, self.mask.data_ptr(),
                                 self.words, self.stream)
        self.states = [after, before]
        self.trace = []   # what the gradient needs of each step
        for _ in range(self.max_new):
            mask, gen_len = self.mask.clone(), self.gen_len.clone()
            alive = self.step()
            self.trace.append((self.hidden, self.logits.clone(), mask, gen_len, self.top.clone(), self.lse.clone()))
            if not alive:
                break
        self.release(torch.ones(n, dtype=torch.uint8, device="cuda"))
        gen, lens = self.gen.cpu().numpy(), self.gen_len.cpu().numpy()
        return [b"".join(self.tok.token_bytes[t] for t in gen[k, :lens[k]]) for k in range(n)]

    def policy_gradient(self, reward):
        """The gradient of sum_k reward[k] * log p(all choices of request k) with
        respect to the model's output weights, under the rules of each step: a
        row of scores for each step and request.  Rows of requests that had
        ended (their masks are empty) get zeros."""
        steps = len(self.trace)
        rows = steps * self.n
        hidden, logits, mask, gen_len, pick, lse = (torch.cat(t) for t in zip(*self.trace))

        def each(t):
            return t.repeat(steps, *[1] * (t.dim() - 1))

        keep = dict(d_logits=logits, d_seen=each(self.seen), d_gen=self.gen, d_gen_start=each(self.gen_start),
                    d_gen_len=gen_len, d_repetition=each(self.repetition), d_frequency=each(self.frequency),
                    d_presence=each(self.presence), d_temperature=each(self.temperature),
                    d_bias_off=torch.arange(rows + 1, device="cuda"), d_bias_id=each(self.bias_id), d_bias=each(self.bias),
                    d_mask=mask, d_pick=pick, d_top=pick, d_lse=lse)
        args = bpe.LogitsArgs(logits_stride=self.V, dtype=bpe.DTYPE_BF16, rows=rows, n_logits=self.V, seen_stride=self.words,
                              mask_stride=self.words, **{k: t.data_ptr() for k, t in keep.items()})
        grad, weight = torch.empty_like(logits), each(reward)
        self.tok.process_logits_backward_device(
            args, bpe.LogitsGradArgs(d_grad_logprob=weight.data_ptr(), d_grad_logits=grad.data_ptr(),
                                     grad_logits_stride=self.V), self.stream)
        return grad.t().float() @ hidden.float(), grad.view(steps, self.n, self.V)


def main():
    tok = bpe.Tokenizer.from_merges_file(os.path.join(ROOT, "data", "vocabs", "gpt2_mixed_50k.merges"), bpe.PATTERN_GPT2)
    prompts = [b"Describe the build as a record.\n", "Une phrase accentuée, s'il vous plaît: ".encode(),
               b"def main():\n    return 42\n" * 40]
    d = Decoder(tok, prompts, *record_grammar())
    for p, out, score in zip(prompts, d.run(), d.score.tolist()):
        print("%-34r -> %s   (log-probability %.2f)" % (p[:30], out.decode(), score))
    w, _ = d.policy_gradient(torch.ones(len(prompts), device="cuda"))
    print("gradient of the output weights: %s, norm %.4f" % (tuple(w.shape), float(w.norm())))


if __name__ == "__main__":
    main()
