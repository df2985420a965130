"""Caches, batches and calls for the attention sub-layer's GPU tests."""
import torch

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


class Cache:
    """A paged cache whose every byte starts as `fill` codes and `scale` scales (127 and 255: NaN, as memory may hold)."""

    def __init__(self, E, n_pages, KH, pt, D, page_stride=0, fill=127, scale=255):
        self.n_pages, self.KH, self.pt, self.D = n_pages, KH, pt, D
        stride = page_stride or KH * pt * D
        self.raw = [torch.full((n_pages * stride,), fill, dtype=torch.uint8, device="cuda") for _ in "kv"]
        self.k, self.v = (torch.as_strided(r, (n_pages, KH, pt, D), (stride, pt * D, D, 1)) for r in self.raw)
        self.ks, self.vs = (torch.full((n_pages, KH), scale, dtype=torch.uint8, device="cuda") for _ in "kv")
        self.desc = E.KvCache(self.raw[0], self.raw[1], self.ks, self.vs, n_pages, KH, pt, D, page_stride)

    def clone_into(self, other):
        for a, b in ((self.k, other.k), (self.v, other.v), (self.ks, other.ks), (self.vs, other.vs)):
            b.copy_(a)

    def tensors(self):
        return self.k, self.v, self.ks, self.vs


def batch(E, table, new, kv, uniform=False, max_rows=None):
    """table [B, pages] int32 (cuda), new and kv lists of ints."""
    start = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    b = E.KvBatch(table, lens, None if uniform else start, len(new), table.shape[1], sum(new),
                  max(new) if max_rows is None else max_rows, table.stride(0))
    b.lens, b.start = lens, start
    return b


def pages_for(kv, pt, n_pages, seed=0, width=None):
    """Pages of each sequence from a shuffled pool; unused entries point outside the cache."""
    need = [-(-n // pt) for n in kv]
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    assert sum(need) <= n_pages
    t = torch.full((len(kv), width or max(1, max(need))), -7, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            t[b, i] = order.pop()
    return t.cuda()


def fill_random(cache, table, kv, seed, spread=2):
    """Random codes (finite) and scales for the tokens of the sequences; everything else stays as it was."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b, n in enumerate(kv):
        for i in range(-(-n // cache.pt)):
            p, m = int(table[b, i]), min(cache.pt, n - i * cache.pt)
            for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
                x = torch.randn((cache.KH, m, cache.D), generator=g, device="cuda") * 60
                codes[p, :, :m] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                scales[p] = 121 + torch.randint(-spread, spread + 1, (cache.KH,), generator=g, device="cuda").to(torch.uint8)


def sequence_tokens(R, cache, table, b, n):
    """k, v [n, KH, D] in 64 bits of the first n tokens of sequence b."""
    out = []
    for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
        pages = table[b, : -(-n // cache.pt)].long()
        x = R.dequant(codes[pages], scales[pages])
        out.append(x.permute(0, 2, 1, 3).reshape(-1, cache.KH, cache.D)[:n])
    return out
