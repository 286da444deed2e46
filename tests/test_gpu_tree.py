"""tree_attention on the GPU against its definition in 64 bits."""
import random

import pytest
import torch

from masked_reference import assert_within
from step_reference import words_of
from tree_reference import reference

pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 0.021, 0.017


def tree_masks(n, rng, reach=9):
    """Ancestors' bits of a random tree's rows."""
    masks = []
    for i in range(n):
        up = rng.randint(max(-1, i - reach), i - 1) if i else -1
        masks.append((masks[up] if up >= 0 else 0) | 1 << i)
    return masks


class Batch:
    """Requests (q_len, context) with trees; blocks that no request holds, the null
    block and slots behind a request's keys hold NaN."""

    def __init__(self, requests, hq, hkv, d, block=16, fp8=False, words=1, seed=0, pad_rows=0, masks=None, mul=2.0):
        rng = random.Random(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_lens = [n for n, _ in requests]
        self.seq_lens = [n + c for n, c in requests]
        self.masks = masks if masks is not None else sum((tree_masks(n, rng) for n in self.q_lens), [])
        self.rows = sum(self.q_lens)
        self.words, self.scale, self.fp8 = words, d ** -0.5, fp8
        need = [-(-n // block) for n in self.seq_lens]
        width = max(need + [1]) + 1
        nb = sum(need) + 4
        ids = list(range(1, nb))
        rng.shuffle(ids)
        tables = [[ids.pop() for _ in range(k)] + [0] * (width - k) for k in need]
        self.tables = torch.tensor(tables, dtype=torch.int32, device="cuda").view(len(requests), width)
        self.kc, self.vc = (self._cache((nb, block, hkv, d), gen, s) for s in (K_SCALE, V_SCALE))
        self.nan = 0x7F if fp8 else float("nan")
        for c in (self.kc, self.vc):
            held = torch.zeros(nb, block, dtype=torch.bool, device="cuda")
            for r, n in enumerate(self.seq_lens):
                t = torch.arange(n, device="cuda")
                held[self.tables[r].long()[t // block], t % block] = True
            c[~held] = self.nan
        self.q = (torch.randn(self.rows + pad_rows, hq, d, generator=gen, device="cuda") * mul).bfloat16()
        self.qsl = torch.tensor([sum(self.q_lens[:i]) for i in range(len(requests) + 1)], dtype=torch.int32, device="cuda")
        self.sl = torch.tensor(self.seq_lens, dtype=torch.int32, device="cuda")
        self.set_masks(self.masks, pad_rows)

    def set_masks(self, masks, pad_rows=0):
        self.masks = masks
        self.m = torch.tensor(words_of(masks, self.words) + [[-1] * self.words] * pad_rows, dtype=torch.int64,
                              device="cuda").view(-1, self.words)

    def _cache(self, shape, gen, scale):
        x = torch.randn(shape, generator=gen, device="cuda")
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if self.fp8 else x.bfloat16()

    def run(self, pa, **kw):
        call, scales = (pa.tree_attention_fp8, (K_SCALE, V_SCALE)) if self.fp8 else (pa.tree_attention, ())
        return call(self.q, self.kc, self.vc, self.qsl, self.sl, self.tables, kw.pop("masks", self.m),
                    kw.pop("max_query_len", max(self.q_lens)), kw.pop("max_seq_len", max(self.seq_lens)), self.scale,
                    *scales, **kw)

    def ref(self):
        s = (K_SCALE, V_SCALE) if self.fp8 else (1.0, 1.0)
        return reference(self.q[:self.rows], self.kc, self.vc, self.tables, self.seq_lens, self.q_lens, self.masks,
                         self.scale, *s)

    def check(self, pa, **kw):
        ws = pa.new_workspace(pa.tree_workspace_size(len(self.q_lens), self.q.shape[0], self.q.shape[1],
                                                     self.kc.shape[2], self.q.shape[2], max(self.seq_lens)), "cuda")
        out = torch.full_like(self.q, 3.5)
        got = self.run(pa, out=out, workspace=ws, **kw)
        assert pa.device_status(ws)[0] == 0
        assert (got[self.rows:] == 3.5).all()
        assert_within(got[:self.rows], *self.ref())
        return got


SHAPES = [  # requests, hq, hkv, d, block, words
    ([(1, 0)], 1, 1, 64, 16, 1),
    ([(1, 6)], 4, 2, 128, 16, 1),
    ([(5, 32), (4, 10), (5, 0), (3, 127)], 4, 2, 64, 16, 1),
    ([(8, 700), (8, 121), (8, 120), (8, 119)], 8, 2, 128, 16, 1),          # nodes across a step's border
    ([(16, 1000), (1, 77), (0, 40), (33, 300)], 32, 8, 128, 16, 1),        # one slot and two
    ([(64, 500), (64, 64), (63, 1), (17, 2000)], 8, 2, 128, 32, 1),        # 256 rows a kv head
    ([(64, 130), (40, 259), (9, 511)], 16, 2, 64, 64, 1),                  # more than one unit a kv head
    ([(130, 300), (7, 65), (200, 90), (256, 0)], 7, 1, 128, 16, 4),        # group 7, long masks
    ([(20, 31), (37, 900), (11, 4)], 10, 2, 64, 16, 1),                    # group 5
    ([(48, 333), (3, 2000)], 48, 3, 128, 16, 1),                           # group 16
    ([(129, 400), (127, 128), (128, 127)], 3, 3, 128, 16, 3),              # group 1: tiles of 128 nodes
    ([(24, 20000), (1, 15)], 8, 2, 128, 16, 1),                            # cut over many CTAs
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_trees(cuda_lib, shape, fp8):
    requests, hq, hkv, d, block, words = SHAPES[shape]
    Batch(requests, hq, hkv, d, block=block, fp8=fp8, words=words, seed=shape, pad_rows=3).check(cuda_lib)
