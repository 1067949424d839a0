"""Float64 CPU oracle of what stands around the decoder layers: the linear in
8-bit integers, the logits' rules with the choice of a token, and the pages of
the 8-bit cache, sequence by sequence.  Test infrastructure only."""
import numpy as np


# ------------------------------------------------------- linear in 8 bits

def quantize8(x):
    """codes int8 and scales of the rows of x (float64 holding bf16 values).  A
    scale is fp32; bf16 / fp32 quotients are at least 2^-33 of their size away
    from a border or on it, so float64 rounds them right."""
    top = np.abs(x).max(-1)
    scale = (top.astype(np.float32) / np.float32(127)).astype(np.float64)
    bad = ~np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x / scale[:, None])
    q[(scale == 0) | bad] = 0
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def linear8(q, s, w, t):
    """(sums, scales): the codes' sums, whole numbers that float64 holds, and what
    each is multiplied with."""
    dot = q.astype(np.float64) @ w.astype(np.float64).T
    return dot, s[:, None] * t[None, :].astype(np.float64)


# ------------------------------------------------------------------ logits

def logits(x, history=None, history_lens=None, prompt_lens=None, repetition=None, frequency=None, presence=None,
           bias_offsets=None, bias_ids=None, bias=None, allowed=None, temperature=None, real=np.float64):
    """The rules, each step rounded to `real`: float64 for their value, float32 for
    the very numbers.  Returns (logits, token, lse, logprob), the last two in
    float64."""
    x = np.array(x, dtype=real)
    B, V = x.shape
    with np.errstate(all="ignore"):
        for b in range(B):
            row = x[b]
            if history is not None:
                n = min(max(int(history_lens[b]), 0), history.shape[1])
                p = 0 if prompt_lens is None else min(max(int(prompt_lens[b]), 0), n)
                count = {}
                for i in range(n):
                    v = int(history[b, i])
                    if 0 <= v < V:
                        count[v] = count.get(v, 0) + (i >= p)
                for v, c in count.items():
                    if repetition is not None:
                        r = real(repetition[b])
                        row[v] = row[v] / r if row[v] > 0 else row[v] * r
                    if c:
                        if frequency is not None:
                            row[v] = row[v] - real(real(frequency[b]) * real(c))
                        if presence is not None:
                            row[v] = row[v] - real(presence[b])
            if bias is not None:
                lo = min(max(int(bias_offsets[b]), 0), len(bias))
                hi = min(max(int(bias_offsets[b + 1]), lo), len(bias))
                for i in range(lo, hi):
                    if 0 <= bias_ids[i] < V:
                        row[bias_ids[i]] = row[bias_ids[i]] + real(bias[i])
            if temperature is not None:
                t = real(temperature[b])
                row *= real(1) / t if t > 0 else real(1)
            if allowed is not None:
                words = allowed[b].astype(np.uint32)
                v = np.arange(V)
                row[(words[v // 32] >> (v % 32).astype(np.uint32)) & 1 == 0] = -np.inf
        token = np.full(B, -1, dtype=np.int64)
        lse, logprob = np.full(B, -np.inf), np.full(B, -np.inf)
        for b in range(B):
            row = x[b].astype(np.float64)
            some = row > -np.inf
            if some.any():
                token[b] = np.flatnonzero(some & (row == row[some].max()))[0]
            if np.isnan(row).any() or np.isposinf(row).any():
                lse[b] = logprob[b] = np.nan
            elif some.any():
                top = row.max()
                log_sum = np.log(np.exp(row - top).sum())
                lse[b], logprob[b] = top + log_sum, -log_sum
    return x, token, lse, logprob


# ------------------------------------------------------------------- pages

class Pool:
    """refs, table, lens as lists; every call does its list one by one."""

    def __init__(self, blocks, slots, most, block):
        self.refs, self.lens, self.block, self.most = [0] * blocks, [0] * slots, block, most
        self.table = [[-1] * most for _ in range(slots)]

    def pages(self, n):
        return -(-n // self.block)

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            if not 0 <= s < len(self.lens):
                continue
            k = max(0, keep[i]) if keep is not None else 0
            for j in range(self.pages(k), self.pages(self.lens[s])):
                if self.table[s][j] >= 0:
                    self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            self.lens[s] = min(self.lens[s], k)

    def fork(self, parents, children):
        lens, table = list(self.lens), [list(r) for r in self.table]
        for i, (f, t) in enumerate(zip(parents, children)):
            if not (0 <= f < len(lens) and 0 <= t < len(lens)) or t in parents or t in children[:i] or lens[t] != 0:
                continue
            n = self.pages(lens[f])
            self.table[t][:n] = table[f][:n]
            for p in table[f][:n]:
                self.refs[p] += 1
            self.lens[t] = lens[f]

    def alloc(self, seqs, new):
        granted, pairs, stop = [0] * len(seqs), [], False
        free = [i for i, r in enumerate(self.refs) if r == 0]
        good = [i for i, s in enumerate(seqs) if 0 <= s < len(self.lens) and s not in seqs[:i] and new[i] >= 0
                and self.lens[s] + new[i] <= self.most * self.block]

        def page(i):   # the page that entry i would write into and others hold
            s = seqs[i]
            p = self.table[s][self.lens[s] // self.block] if self.lens[s] % self.block and new[i] else -1
            return p if p >= 0 and refs[p] > 1 else -1
        refs = list(self.refs)
        shared = {i: page(i) for i in good}
        for i in good:
            s, old = seqs[i], self.lens[seqs[i]]
            p = shared[i]
            others = [j for j in good if p >= 0 and shared[j] == p]
            copy = p >= 0 and not (len(others) == refs[p] and others[-1] == i)
            need = self.pages(old + new[i]) - self.pages(old) + copy
            stop = stop or need > len(free)
            if stop:
                continue
            mine, free = free[:need], free[need:]
            at = old // self.block if copy else self.pages(old)
            if copy:
                pairs.append((p, mine[0]))
                self.refs[p] -= 1
            for j, q in enumerate(mine):
                self.table[s][at + j] = q
                self.refs[q] = 1
            self.lens[s] = old + new[i]
            granted[i] = 1
        return granted, pairs

    def compact(self):
        live = [i for i, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [i for i in range(n) if self.refs[i] <= 0]
        pairs = list(zip([i for i in live if i >= n], holes))
        moved = [i if r > 0 else -1 for i, r in enumerate(self.refs)]
        for f, t in pairs:
            moved[f], self.refs[t], self.refs[f] = t, self.refs[f], 0
        for s, row in enumerate(self.table):
            for j in range(self.pages(self.lens[s])):
                row[j] = moved[row[j]]
        return pairs, moved
