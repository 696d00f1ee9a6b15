"""kvd_paged_append against its definition: where rows go, rotated keys and queries, strides,
tokens of no row, lengths and pages that do not fit."""

import numpy as np
import pytest
import torch

import ref64_serving as ref
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Case:
    """rows: (new tokens, positions before them)."""

    def __init__(self, rows, hq, hk, page, dtype=torch.float16, order="head", seed=0, lead=0,
                 trail=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.hq, self.hk, self.page = rows, hq, hk, page
        need = [-(-max(n + s, 1) // page) for n, s in rows]
        self.n_pages = sum(need) + 2
        shape = (self.n_pages, hk, page, 64) if order == "head" else (self.n_pages, page, hk, 64)
        self.pools = []
        for _ in "kv":
            t = torch.randn(shape, generator=g, device="cuda").to(dtype)
            self.pools.append(t if order == "head" else t.transpose(1, 2))
        perm = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(rows), max(need)), -9, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = perm[at:at + k]
            at += k
        starts = [lead]
        for n, _ in rows:
            starts.append(starts[-1] + n)
        self.T, self.host_starts = starts[-1] + trail, starts
        i32 = dict(dtype=torch.int32, device="cuda")
        self.starts = torch.tensor(starts, **i32)
        self.lens = torch.tensor([s for _, s in rows], **i32)
        self.qkv = torch.randn(self.T, hq + 2 * hk, 64, generator=g, device="cuda").to(dtype)
        self.before = [t.clone() for t in self.pools]

    def run(self, spec=None, with_q=True, **kw):
        import kv_cached_decode_gb300 as kvd

        hq, hk = self.hq, self.hk
        self.lens_out = torch.full_like(self.lens, -77)
        self.q_out = torch.full((self.T, hq, 64), 5.0, dtype=self.qkv.dtype, device="cuda")
        kvd.kvd_paged_append(
            kvd.make_paged_cache(*self.pools, self.table), self.qkv[:, hq:hq + hk],
            self.qkv[:, hq + hk:], self.starts, self.lens, lens_out=self.lens_out,
            q=self.qkv[:, :hq] if with_q else None, q_out=self.q_out if with_q else None,
            rope=None if spec is None else kvd.make_rope(**spec), **kw)
        torch.cuda.synchronize()

    def check(self, spec=None, with_q=True, skip=(), lost=()):
        """skip: rows left as they are; lost: (row, position) whose page is outside the pool."""
        hq, hk, page = self.hq, self.hk, self.page
        k, v = (t.clone() for t in self.before)
        q = torch.full_like(self.q_out, 5.0)
        size_k = torch.zeros(k.shape, dtype=torch.float64)
        want_k, want_q = k.double().cpu(), q.double().cpu()
        size_q = torch.zeros_like(want_q)
        table, most = self.table.cpu(), 0
        for b, (n, s) in enumerate(self.rows):
            if b in skip:
                continue
            for j in range(n):
                t, pos = self.host_starts[b] + j, s + j
                row = self.qkv[t].double().cpu().numpy()
                most = max(most, pos)
                turned, size = (row, np.zeros_like(row)) if spec is None else ref.rotate(
                    row, np.full(row.shape[0], pos), spec)
                if with_q:
                    want_q[t] = torch.from_numpy(turned[:hq])
                    size_q[t] = torch.from_numpy(size[:hq])
                if (b, pos) in lost:
                    continue
                pg = int(table[b, pos // page])
                want_k[pg, :, pos % page] = torch.from_numpy(turned[hq:hq + hk])
                size_k[pg, :, pos % page] = torch.from_numpy(size[hq:hq + hk])
                v[pg, :, pos % page] = self.qkv[t, hq + hk:]
        assert torch.equal(self.pools[1], v)
        for got, want, size in ((self.pools[0], want_k, size_k), (self.q_out, want_q, size_q)):
            got, want, size = got.double().cpu().numpy(), want.numpy(), size.numpy()
            tol = np.where(size > 0, ref.rotation_bound(want, size, self.qkv.dtype, most), 0.0)
            bad = ~(np.abs(got - want) <= tol)
            assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist())
        assert self.lens_out.tolist() == [s if b in skip else s + n
                                          for b, (n, s) in enumerate(self.rows)]


ROWS = [(1, 0), (5, 14), (0, 9), (33, 60), (2, 0), (1, 100)]
SPECS = [None, dict(), dict(rot_dim=32, interleaved=True), dict(rot_dim=48, magnitude=0.5),
         dict(scaling="ramp", factor=16.0, original_len=64, low=1.0, high=8.0)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("spec", SPECS, ids=range(len(SPECS)))
def test_rows_and_rotations(dtype, spec):
    c = Case(ROWS, 8, 2, 16, dtype)
    c.run(spec)
    c.check(spec)


@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("hq,hk", [(1, 1), (15, 5), (20, 20)])
def test_pages_and_heads(page, order, hq, hk):
    c = Case(ROWS, hq, hk, page, order=order, seed=page)
    c.run(dict())
    c.check(dict())


def test_many_tokens_and_rows():
    c = Case([(700, 3), (1, 0), (300, 500)] + [(1, i) for i in range(100)], 3, 1, 16, lead=3,
             trail=4)
    c.run(dict())
    c.check(dict())


def test_without_queries_and_tokens_of_no_row():
    c = Case(ROWS, 4, 2, 16, lead=7, trail=11)
    c.run(None, with_q=False)
    c.check(None, with_q=False)


def test_queries_in_place():
    import kv_cached_decode_gb300 as kvd

    c = Case(ROWS, 4, 2, 16)
    c.run(dict())
    want = c.q_out.clone()
    q = c.qkv[:, :4].contiguous()
    kvd.kvd_paged_append(kvd.make_paged_cache(*c.pools, c.table), c.qkv[:, 4:6], c.qkv[:, 6:],
                         c.starts, c.lens, q=q, q_out=q, rope=kvd.make_rope())
    torch.cuda.synchronize()
    assert torch.equal(q, want)


def test_lengths_that_do_not_fit():
    for row, s in ((1, -1), (3, 1 << 20), (0, (1 << 31) - 1)):
        c = Case(ROWS, 4, 2, 16)
        c.lens[row] = s
        err = new_err()
        c.run(dict(), dev_err=err)
        rows = list(c.rows)
        rows[row] = (c.rows[row][0], s)
        c.rows = rows
        c.check(dict(), skip=(row,))
        assert int(err) == 16
    c = Case(ROWS, 4, 2, 16)  # the last row ends behind the packed tokens
    c.starts[len(ROWS)] += 1
    err = new_err()
    c.run(dict(), dev_err=err)
    c.check(dict(), skip=(len(ROWS) - 1,))
    assert int(err) == 16


def test_pages_outside_the_pool():
    for bad in (-1, 1 << 30, -(1 << 31)):
        c = Case(ROWS, 4, 2, 16)
        c.table[3, 5] = bad  # positions 80 .. 92 of row 3
        err = new_err()
        c.run(dict(), dev_err=err)
        c.check(dict(), lost=[(3, p) for p in range(80, 96)])
        assert int(err) == 17


def test_no_tokens():
    c = Case([(0, 5), (0, 0)], 4, 2, 16, trail=0)
    c.run(dict())
    c.check(dict())


def test_same_bits_as_the_rotation_alone():
    import kv_cached_decode_gb300 as kvd

    for spec in SPECS[1:]:
        c = Case([(40, 1000)], 6, 2, 16, torch.bfloat16)
        c.run(spec)
        x = c.qkv[:, :6].transpose(0, 1)[None]  # [1, heads, tokens, 64]
        y = torch.empty(1, 6, 40, 64, dtype=torch.bfloat16, device="cuda")
        kvd.kvd_rope_scaled(x, q_out=y, rope=kvd.make_rope(**spec), pos0=c.lens)
        torch.cuda.synchronize()
        assert torch.equal(y[0].transpose(0, 1), c.q_out)
