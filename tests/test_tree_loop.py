"""A serving loop that drafts trees: the accepted path is moved together in the cache and in the sums, what was
drafted besides is forgotten, and the cache stays within a budget."""
import types

import pytest
import torch

import exact_attention_blackwell_gb300 as fa
import paged_model as pm
import rope_model as rm
from test_evict import bits, i32
from test_evict import model as evict_model
from test_weights import check as check_weights
from test_weights import reference as weights_reference

pytestmark = pytest.mark.gpu


class Loop:
    """The caller's program."""

    def __init__(self, B, H, Hkv, d, page, keep, recent, room, layers, seed):
        self.B, self.H, self.Hkv, self.d, self.page = B, H, Hkv, d, page
        self.keep, self.recent, self.layers = keep, recent, layers
        cols = pm.pages_of(room, page)
        pool = B * cols + 1
        self.k, self.v = (torch.full((layers, pool, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.refs, self.table, self.lens = i32([0] * pool), i32([[-1] * cols] * B), i32([0] * B)
        self.sums = torch.zeros((layers, B, Hkv, cols * page), device="cuda")
        self.inv_freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()

    def draft(self, qkv, grown, cu, positions, max_new, mask):
        """All drafted tokens through every layer -> (the lengths with them, [(q, lse)])."""
        held, _ = fa.cache_resize(self.refs, self.k, self.v, self.table, self.lens, self.lens + grown)
        out = []
        for l in range(self.layers):
            q, k, v = qkv[l].split([self.H, self.Hkv, self.Hkv], 1)
            q = fa.cache_append_rope(q, k, v, self.k[l], self.v[l], self.table, self.lens, cu, self.inv_freq, positions)
            o, lse = fa.attention_fwd_paged(q, self.k[l], self.v[l], self.table, self.lens, cu, max_new, tree_mask=mask)
            fa.attention_weights_paged(q, self.k[l], self.table, self.lens, cu, max_new, lse, self.sums[l], tree_mask=mask)
            out.append((q, o, lse))
        return held, out

    def accept(self, held, accepted, n_accepted):
        """The path's rows move together, its sums with them, and the others' are cleared."""
        lens = fa.cache_compact(self.k, self.v, self.table, self.lens, accepted, n_accepted)
        places = torch.arange(self.sums.shape[-1], device="cuda")
        i = (places[None] - self.lens[:, None]).clamp(0, max(accepted.shape[1] - 1, 0)).long()  # of the path
        source = torch.where((places >= self.lens[:, None]) & (places < lens[:, None]),
                             self.lens[:, None].long() + torch.gather(accepted.long(), 1, i), places)
        source = source.clamp(max=self.sums.shape[-1] - 1)[None, :, None].expand_as(self.sums)
        self.sums.copy_(torch.gather(self.sums, -1, source) * (places < lens[:, None])[None, :, None])
        lens, _ = fa.cache_resize(self.refs, self.k, self.v, self.table, held, lens)
        self.lens = lens

    def evict(self):
        lens, kept = fa.cache_evict(self.refs, self.k, self.v, self.table, self.lens, self.sums, self.keep, self.recent)
        self.lens, _ = fa.cache_resize(self.refs, self.k, self.v, self.table, self.lens, lens)
        return kept

    def view(self, layer, lens, new):
        """What the models ask for, of one layer (None: all)."""
        table = self.table.tolist()
        s = types.SimpleNamespace(lens=lens, new=new, page=self.page, Hkv=self.Hkv, d=self.d, B=self.B, table=table, total=sum(new))
        s.k_pages, s.v_pages = (x.cpu() if layer is None else x[layer] for x in (self.k, self.v))
        s.place = lambda b, pos: (table[b][pos // self.page], pos % self.page)
        s.cu = [sum(new[:b]) for b in range(self.B + 1)]
        return s


@pytest.mark.parametrize("B,H,Hkv,d,page,most", [(3, 4, 2, 64, 16, 9), (2, 16, 2, 128, 32, 40), (2, 4, 4, 256, 16, 12)])
def test_trees_are_drafted_accepted_and_evicted(B, H, Hkv, d, page, most):
    keep, recent = 50, 8
    loop = Loop(B, H, Hkv, d, page, keep, recent, room=keep + 6 * most + 40, layers=2, seed=1)
    g = torch.Generator().manual_seed(d)
    # for each layer, sequence and kv head: the sums of the places it holds, in 64 bits, and what they may be off by
    sums = torch.zeros(loop.sums.shape, dtype=torch.float64)
    room = torch.zeros_like(sums)
    at = [0] * B  # the next position
    cut = 0
    for step in range(8):
        new = [int(torch.randint(0, most + 1, (1,), generator=g)) for _ in range(B)]
        new[step % B] = most
        if step == 0:  # the prompts, which are chains
            new = [60 - 7 * b for b in range(B)]
        limit = max(new)
        lens = loop.lens.tolist()
        mask, seen = pm.tree_masks(new, 1, seed=step)
        if step == 0:
            seen = [set(range(i + 1)) for n in new for i in range(n)]
            mask = pm.pack_masks(seen, 1)
        s = loop.view(None, lens, new)
        depth = [at[b] + len(seen[s.cu[b] + i]) - 1 for b in range(B) for i in range(new[b])]
        qkv = torch.randn((2, sum(new), H + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
        before = loop.sums.clone()
        held, out = loop.draft(qkv, i32(new), i32(s.cu), i32(depth), limit, mask.cuda())
        torch.cuda.synchronize()
        assert held.tolist() == [a + n for a, n in zip(lens, new)] and fa.fa_last_device_status() == fa.FA_OK
        angle = rm.angles(torch.tensor(depth), loop.inv_freq.cpu(), None)
        for l in range(2):
            rm.check_forward(out[l][0], qkv[l][:, :H], None, angle, False, what=f"step {step}")
            s = loop.view(l, lens, new)
            ref = weights_reference(s, out[l][0], out[l][2], before[l], seen)
            check_weights(s, loop.sums[l], ref, before[l], f"step {step} layer {l}")
            # the model's own sums grow by what the call adds
            add, off = weights_reference(s, out[l][0], out[l][2], torch.zeros_like(before[l]), seen)
            sums[l] += add
            room[l] += off + 2.0**-23 * sums[l]
        # one drafted token's path is accepted in each sequence (none where nothing was drafted)
        pick = [new[b] - 1 if step % 3 == 0 else int(torch.randint(0, max(new[b], 1), (1,), generator=g)) for b in range(B)]
        paths = [sorted(seen[s.cu[b] + pick[b]]) if new[b] else [] for b in range(B)]
        width = max(len(p) for p in paths)
        rows = [[loop.view(None, lens, new).place(b, lens[b] + j) for j in paths[b]] for b in range(B)]
        k, v, drafted = loop.k.clone(), loop.v.clone(), loop.sums.clone()
        loop.accept(held, i32([p + [-1] * (width - len(p)) for p in paths]), i32([len(p) for p in paths]))
        torch.cuda.synchronize()
        kept_lens = [a + len(p) for a, p in zip(lens, paths)]
        assert loop.lens.tolist() == kept_lens
        for b in range(B):
            source = list(range(lens[b])) + [lens[b] + j for j in paths[b]]
            assert torch.equal(loop.sums[:, b, :, : kept_lens[b]], drafted[:, b][:, :, source])
            for table in (sums, room):
                table[:, b, :, : kept_lens[b]] = table[:, b][:, :, source].clone()
                table[:, b, :, kept_lens[b] :] = 0
            for i, (page_from, row_from) in enumerate(rows[b]):
                page_to, row_to = loop.view(None, lens, new).place(b, lens[b] + i)
                assert torch.equal(loop.k[:, page_to, row_to], k[:, page_from, row_from])
                assert torch.equal(loop.v[:, page_to, row_to], v[:, page_from, row_from])
        # nothing of what was not accepted is left
        behind = torch.arange(sums.shape[-1]) >= torch.tensor(kept_lens)[:, None]
        assert (loop.sums.cpu()[behind[None, :, None].expand(loop.sums.shape)] == 0).all()
        assert ((loop.sums.cpu().double() - sums).abs() <= room + 2.0**-126).all(), f"step {step}"
        at = [a + len(p) for a, p in zip(at, paths)]
        if step % 2:
            s = loop.view(None, kept_lens, [0] * B)
            want = evict_model(s, loop.sums, keep, recent)
            kept = loop.evict()
            torch.cuda.synchronize()
            assert loop.lens.tolist() == want[3] and torch.equal(kept.cpu(), want[4]) and torch.equal(loop.sums.cpu(), want[2])
            assert torch.equal(bits(loop.k.cpu()), bits(want[0])) and torch.equal(bits(loop.v.cpu()), bits(want[1]))
            for b in range(B):
                n = loop.lens.tolist()[b]
                if kept_lens[b] > keep:
                    cut += 1
                    for table in (sums, room):
                        table[:, b, :, :n] = torch.gather(table[:, b], -1, want[4][:, b].long())
                        table[:, b, :, n:] = 0
            assert int((loop.refs > 0).sum()) == sum(pm.pages_of(n, page) for n in loop.lens.tolist())
    assert cut >= B
