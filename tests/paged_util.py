"""A packed ragged batch over a paged cache, for the GPU tests."""

import torch

import ref64
import ref64_serving as ref


class Batch:
    """rows: (new tokens, length with them) per row. lead, trail: packed tokens of no row."""

    def __init__(self, rows, hq, hk, page, dtype=torch.float16, order="head", seed=0, lead=0,
                 trail=0, spare=3, extra_width=2, peak=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.hq, self.hk, self.page, self.dtype = rows, hq, hk, page, dtype
        need = [-(-max(x, 0) // page) for _, x in rows]
        self.n_pages = sum(need) + spare
        shape = (self.n_pages, hk, page, 64) if order == "head" else (self.n_pages, page, hk, 64)
        nan = lambda: torch.full(shape, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
        self.k, self.v = nan(), nan()
        if order != "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        perm = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        width = max(need + [1]) + extra_width
        self.table = torch.full((len(rows), width), 1 << 30, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = perm[at:at + k]
            at += k
        # values up to each row's length; the rest of every page stays NaN
        for b, (_, length) in enumerate(rows):
            for i in range(need[b]):
                m = min(page, length - i * page)
                for t in (self.k, self.v):
                    t[self.table[b, i].long(), :, :m] = torch.randn(
                        hk, m, 64, generator=g, device="cuda").to(dtype)
        starts = [lead]
        for n, _ in rows:
            starts.append(starts[-1] + n)
        self.T = starts[-1] + trail
        i32 = dict(dtype=torch.int32, device="cuda")
        self.starts, self.lens = torch.tensor(starts, **i32), torch.tensor([x for _, x in rows],
                                                                          **i32)
        self.q = (torch.randn(self.T, hq, 64, generator=g, device="cuda") * peak).to(dtype)
        self.host_starts = starts

    def cache(self):
        import kv_cached_decode_gb300 as kvd

        return kvd.make_paged_cache(self.k, self.v, self.table)

    def workspace(self, max_new):
        import kv_cached_decode_gb300 as kvd

        return kvd.new_workspace(kvd.kvd_workspace_size(
            kvd.KVD_OP_PAGED_ATTN, len(self.rows), self.hq, self.hk, 1, max_new))

    def most_new(self):
        return max([n for n, _ in self.rows] + [1])

    def attend(self, out=None, max_new=None, workspace=None, scale=0.125, q=None, **kw):
        import kv_cached_decode_gb300 as kvd

        out = torch.full_like(self.q, 7.0) if out is None else out
        m = max_new or self.most_new()
        ws = self.workspace(m) if workspace is None else workspace
        kvd.kvd_paged_attn(self.q if q is None else q, self.cache(), out, ws, self.starts,
                           self.lens, max_new=m, scale=scale, **kw)
        return out

    def check(self, out, scale=0.125, skip=(), untouched=7.0):
        """Every row against the 64-bit form; packed tokens of no row (and rows in `skip`)
        untouched."""
        torch.cuda.synchronize()
        seen = torch.zeros(self.T, dtype=torch.bool)
        table = self.table.cpu()
        for b, (n, length) in enumerate(self.rows):
            if n <= 0 or b in skip:
                continue
            s = self.host_starts[b]
            seen[s:s + n] = True
            k, v = ref.paged_rows(self.k, self.v, table, b, length)
            want, mag, size, low = ref.chunk_attention(self.q[s:s + n].double(), k, v, scale)
            tol = ref64.attention_bound(want, mag, size, self.dtype,
                                        floor=low if self.dtype == torch.float16 else 0.0)
            bad = ~((out[s:s + n].double() - want).abs() <= tol)
            assert not bad.any(), (b, int(bad.sum()), bad.nonzero()[0].tolist(),
                                   out[s:s + n][bad][:4].tolist(), want[bad][:4].tolist())
        assert (out[~seen.to(out.device)] == untouched).all()
