"""Seeded batches for the dense latent attentions and their definitions in 64 bits.

Cache rows that no query may see (behind a sequence's kv_len, between sequences,
spare pages) hold NaN, so anything that reaches a result from there shows.

Tolerances.  With p the probabilities and A = sum p |v| elementwise, the kernels
round each probability and the result to bf16 (2^-8 relative each at most), and
their scores are fp32 sums of K exact products: off by at most
K * 2^-24 * scale * sum |q k| =: e, which moves a probability by a factor within
1 +- 2 e (its own score and the normaliser's).  So
    |out - exact| <= A * (2^-8 + 2 e + 2^-18) + 2^-8 |exact|
(2^-18 for exp2, the row sums and the merge of pieces), |lse - exact| <= e +
2^-20 (1 + |lse|).  The 2-norm over a result of independent roundings stays below 2^-8.
"""

import numpy as np
import torch

import long_context_sparse_lightning_b200 as dsa

BF16_HALF = 2.0 ** -8


class Case:
    def __init__(self, q_len, kv_len, heads, page=0, seed=0, q_dim=576, scale=192 ** -0.5, pad_rows=0, prefix=0,
                 mag=1.0):
        g = torch.Generator().manual_seed(seed)
        self.q_len, self.kv_len, self.heads, self.page, self.scale = list(q_len), list(kv_len), heads, page, scale
        n = len(q_len)
        self.rows = sum(q_len)
        total_q = self.rows + pad_rows
        cu = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.at = []                                     # cache row of every position of every sequence
        if page:
            whole = prefix // page
            blocks = [-(-k // page) for k in kv_len]
            shared = min([whole] + [k // page for k in kv_len]) if prefix else 0
            pages = shared + sum(b - shared for b in blocks) + 3
            order = torch.randperm(pages, generator=g).numpy().astype(np.int32)
            table = np.full((n, max(max(blocks), 1)), -1, np.int32)
            table[:, :shared] = order[:shared]
            nxt = shared
            for b in range(n):
                for i in range(shared, blocks[b]):
                    table[b, i] = order[nxt]
                    nxt += 1
                s = np.arange(kv_len[b])
                self.at.append(table[b][s // page].astype(np.int64) * page + s % page)
            self.total_keys = pages * page
            self.start = None
            self.table = torch.from_numpy(table).cuda()
        else:
            start, at = [], 2
            for k in kv_len:
                start.append(at)
                self.at.append(at + np.arange(k))
                at += k + 5
            self.total_keys = max(at - 5, max(s + k for s, k in zip(start, kv_len)), 1)
            self.start = torch.tensor(start, dtype=torch.int64).cuda()
            self.table = None
        self.cache = torch.full((self.total_keys, 576), float("nan"), dtype=torch.bfloat16)
        self.used = np.unique(np.concatenate(self.at)) if sum(kv_len) else np.zeros(0, np.int64)
        self.cache[self.used] = (torch.randn((len(self.used), 576), generator=g) * mag).to(torch.bfloat16)
        if prefix and page:                              # the partial page behind the shared ones: equal rows
            for b in range(1, n):
                m = min(prefix, kv_len[b], kv_len[0])
                self.cache[self.at[b][:m]] = self.cache[self.at[0][:m]].clone()
        self.q = (torch.randn((total_q, heads, q_dim), generator=g) * mag).to(torch.bfloat16)
        self.g = g
        self.cu_q = torch.from_numpy(cu).cuda()
        self.kv = torch.tensor(kv_len, dtype=torch.int32).cuda()
        self.batch = dsa.Batch(self.cu_q, self.kv, self.start, total_q, max(max(q_len), 1), max(kv_len),
                               self.total_keys, block_table=self.table, page_size=page)

    def outputs(self, dim):
        out = torch.full((self.batch.total_q, self.heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.batch.total_q, self.heads), 7.0, dtype=torch.float32, device="cuda")
        return out, lse

    def dense(self, prefix=None, ws=None, check=True):
        out, lse = self.outputs(512)
        op = dsa.OP_DENSE_MLA if prefix is None else dsa.OP_PREFIX_MLA
        if ws is None:
            ws = dsa.workspace(op, self.batch, n_heads=self.heads)
        if prefix is None:
            dsa.dense_mla(self.batch, self.q.cuda(), self.cache.cuda(), self.scale, out, lse, ws)
        else:
            dsa.prefix_mla(self.batch, prefix, self.q.cuda(), self.cache.cuda(), self.scale, out, lse, ws)
        if check:
            dsa.check_device_error(ws)
        return out.cpu(), lse.cpu()

    def exact(self, keys_values):
        """out, lse, A and e in 64 bits; keys_values(b) -> keys [kv, heads, d], values [kv, heads, dv] of sequence b."""
        outs, lses, As, es = [], [], [], []
        row = 0
        for b, (n, kv) in enumerate(zip(self.q_len, self.kv_len)):
            if n == 0:
                continue
            q = self.q[row:row + n].double()
            k, v = keys_values(b)
            x = torch.einsum("ihd,shd->his", q, k) * self.scale
            sees = torch.arange(kv)[None, :] <= (kv - n + torch.arange(n))[:, None]
            x = x.masked_fill(~sees, float("-inf"))
            p = torch.softmax(x, -1)
            outs.append(torch.einsum("his,shd->ihd", p, v))
            As.append(torch.einsum("his,shd->ihd", p, v.abs()))
            lses.append(torch.logsumexp(x, -1).T)
            mag = torch.einsum("ihd,shd->hi", q.abs(), k.abs().amax(0, keepdim=True)).T * self.scale
            es.append(mag * q.shape[-1] * 2.0 ** -24)
            row += n
        return torch.cat(outs), torch.cat(lses), torch.cat(As), torch.cat(es)

    def exact_dense(self):
        def kv(b):
            c = self.cache[self.at[b]].double()[:, None, :].expand(-1, self.heads, -1)
            return c, c[..., :512]
        return self.exact(kv)


def check(out, lse, exact, rows):
    o, z, A, e = exact
    got = out[:rows].double()
    assert torch.isfinite(got).all()
    tol = A * (BF16_HALF + 2 * e[..., None] + 2.0 ** -18) + BF16_HALF * o.abs()
    d = (got - o).abs()
    assert (d <= tol).all(), f"worst {(d / tol).max()}"
    assert d.norm() <= BF16_HALF * o.norm(), f"2-norm {d.norm() / o.norm()}"
    dz = (lse[:rows].double() - z).abs()
    assert (dz <= e + 2.0 ** -20 * (1 + z.abs())).all(), f"lse {dz.max()}"
    # rows behind the last sequence are left as they were
    assert (out[rows:] == 7.0).all() and (lse[rows:] == 7.0).all()


def _definition(q, k, v, scale):
    """One row in 64 bits over the keys it sees, every product taken (0 x inf too): out, lse."""
    x = (q * k).sum(-1) * scale
    p = torch.softmax(x, -1)
    return (p[:, None] * v).sum(0), torch.logsumexp(x, -1)


def compare_nonfinite(c, out, lse, keys_values):
    """Values or keys that are not finite: NaN exactly where it has to be, and the roundings' 2-norm over the rest;
    keys_values(b, h) -> keys, values of head h.  Returns how many outputs are NaN."""
    row, err, ref, nan_dims = 0, 0.0, 0.0, 0
    for b, (n, kv) in enumerate(zip(c.q_len, c.kv_len)):
        for i in range(n):
            see = kv - n + i + 1
            for h in range(c.heads):
                k, v = keys_values(b, h)
                want, z = _definition(c.q[row, h].double(), k[:see], v[:see], c.scale)
                got = out[row, h].double()
                bad = ~torch.isfinite(want)          # an infinite value of weight > 0 is NaN too
                assert torch.equal(torch.isnan(got), bad), (row, h, torch.isnan(got).sum(), bad.sum())
                assert torch.isfinite(got[~bad]).all()
                err += float((got - want)[~bad].square().sum())
                ref += float(want[~bad].square().sum())
                if torch.isfinite(z):
                    assert abs(float(lse[row, h]) - float(z)) <= 1e-3 * (1 + abs(float(z)))
                else:
                    assert torch.isnan(lse[row, h]) or not bad.all()
                nan_dims += int(bad.sum())
            row += 1
    assert err ** 0.5 <= 2.0 ** -8 * ref ** 0.5
    return nan_dims
