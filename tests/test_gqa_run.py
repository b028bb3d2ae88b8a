"""The operators of layers with grouped heads run together, as a server uses them: pages and slots for prompts that
enter, the write of their keys and values, prompt attention over the packed rows, then decode steps -- pages, write,
attention over the cache -- whose results have to be what prompt attention gives for the same tokens; requests that
end, and others that take their pages.  A latent layer reads the same page table."""
import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


class Server:
    def __init__(self, B, H, K, D, fp8, num_pages, max_pages, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.K, self.D, self.fp8, self.P = B, H, K, D, fp8, num_pages
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.seq, self.table = i32(B), torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(num_pages, generator=self.g, device="cuda").to(torch.int32)
        self.count = torch.tensor([num_pages], dtype=torch.int32, device="cuda")
        shape = (num_pages, K, 64, D)
        dt = torch.uint8 if fp8 else torch.bfloat16
        self.caches = [torch.full(shape, 0x7f, device="cuda").to(dt) for _ in range(2)]
        self.scales = [torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2)]
        self.k, self.v = ([torch.empty((0, K, D), dtype=torch.bfloat16, device="cuda") for _ in range(B)] for _ in range(2))

    def add(self, change):
        """One call of each for `change` tokens a request: (offsets, queries, outputs of prompt attention)."""
        B, H, K, D = self.B, self.H, self.K, self.D
        n = [max(0, c) for c in change]
        T = sum(n)
        rows = torch.randn(T, (H + 2 * K) * D, generator=self.g, device="cuda").to(torch.bfloat16)
        q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([H * D, K * D, K * D], dim=1))
        cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        slots = torch.empty(T, dtype=torch.int32, device="cuda")
        ch = torch.tensor(change, dtype=torch.int32, device="cuda")
        api.dsa_pages_update(ch, self.seq, self.table, self.free, self.count, cu, slots)
        if self.fp8:
            api.dsa_kv_write_fp8(k, v, slots, self.caches[0], self.scales[0], self.caches[1], self.scales[1])
        else:
            api.dsa_kv_write(k, v, slots, *self.caches)
        at = 0
        for r, c in enumerate(change):
            if c < 0:
                self.k[r], self.v[r] = self.k[r][:0], self.v[r][:0]
            else:
                self.k[r], self.v[r] = torch.cat([self.k[r], k[at:at + c]]), torch.cat([self.v[r], v[at:at + c]])
                at += c
        return cu, q, max(n)

    def prompt(self, cu, q, most):
        """Prompt attention of the last tokens over the packed keys of all."""
        cu_k = torch.tensor([0] + list(torch.tensor([len(x) for x in self.k]).cumsum(0)), dtype=torch.int32, device="cuda")
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        api.dsa_gqa_prefill(q, torch.cat(self.k), torch.cat(self.v), cu, cu_k, out, most, self.D ** -0.5)
        return out

    def decode(self, q, nq):
        desc = api.make_desc(self.seq, self.table, nq, self.H, 1, self.P)
        ws = torch.empty(api.dsa_gqa_decode_workspace_bytes(desc, self.K, self.D), dtype=torch.uint8, device="cuda")
        out = torch.empty((self.B * nq, self.H, self.D), dtype=torch.bfloat16, device="cuda")
        q = q.contiguous()
        if self.fp8:
            api.dsa_gqa_decode_fp8kv(desc, q, self.caches[0], self.scales[0], self.caches[1], self.scales[1], out, ws, self.D ** -0.5)
        else:
            api.dsa_gqa_decode(desc, q, *self.caches, out, ws, self.D ** -0.5)
        return out


def _near(a, b, fp8):
    """Both round probabilities (2^-8) and outputs (2^-8) of unit values' means; FP8 rows are off by 2^-4 of their
    values.  Compared by their norms."""
    err = (a.float() - b.float()).norm() / b.float().norm()
    assert err <= (0.06 if fp8 else 0.01), err


@pytest.mark.parametrize("H,K,D,fp8,nq", [(32, 8, 128, False, 1), (32, 8, 128, True, 1), (10, 2, 64, False, 2),
                                          (20, 4, 128, True, 2), (48, 1, 128, False, 1), (64, 2, 128, True, 2)])
def test_prompts_then_steps(H, K, D, fp8, nq):
    lens = [130, 64, 401, 1, 63, 700]
    s = Server(len(lens), H, K, D, fp8, 40, 14, seed=H + nq)
    cu, q, most = s.add(lens)
    assert s.seq.tolist() == lens and s.count.item() == 40 - sum(-(-n // 64) for n in lens)
    s.prompt(cu, q, most)
    for step in range(4):
        cu, q, most = s.add([nq] * len(lens))
        _near(s.decode(q, nq), s.prompt(cu, q, most), fp8)
    # two requests end, one of them is entered again at once and gets pages in the next call
    change = [nq] * len(lens)
    change[1] = change[2] = -1
    s.add(change)
    held = [-(-n // 64) for n in s.seq.tolist()]
    assert s.seq.tolist()[1] == 0 and s.count.item() == 40 - sum(held)
    s.add([0, 200, 0, 0, 0, 0])
    used = [p for r, n in enumerate(s.seq.tolist()) for p in s.table[r, :-(-n // 64)].tolist()]
    assert len(set(used)) == len(used) and not set(used) & set(s.free[:s.count.item()].tolist())
    cu, q, most = s.add([nq, nq, 0, nq, nq, nq])
    got = s.decode(torch.cat([q[:2 * nq], q[:nq], q[2 * nq:]]), nq)
    assert (got[2 * nq:3 * nq] == 0).all()                 # the row without a request
    _near(torch.cat([got[:2 * nq], got[3 * nq:]]), s.prompt(cu, q, most), fp8)
    assert api.dsa_get_device_error() == 0


def test_a_latent_layer_reads_the_same_table():
    """dsa_cache_write and dense latent attention over the pages that dsa_pages_update handed out."""
    s = Server(3, 16, 4, 128, False, 20, 8, seed=1)
    s.add([100, 300, 64])
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *x: torch.randn(*x, generator=g, device="cuda").to(torch.bfloat16)
    latent = torch.zeros((20 * 64, 576), dtype=torch.bfloat16, device="cuda")
    k8, ks = torch.zeros((20 * 64, 128), dtype=torch.uint8, device="cuda"), torch.ones(20 * 64, device="cuda")
    rows = {0: [], 1: [], 2: []}
    for step in range(3):
        s.add([1, 1, 1])
        new = rnd(3, 576)
        api.dsa_cache_write(api.make_desc(s.seq, s.table, 1, 16, 1, 20), new, rnd(3, 128), latent, k8, ks)
        for r in range(3):
            rows[r].append(new[r])
    for r, n in enumerate(s.seq.tolist()):
        pos = torch.arange(n - 3, n, device="cuda")
        at = s.table[r, pos // 64].long() * 64 + pos % 64
        assert torch.equal(latent[at], torch.stack(rows[r]))
    assert api.dsa_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_step(fp8):
    """A decode step -- pages, write, attention -- captured once and replayed: lengths, table and caches grow in place."""
    s = Server(5, 32, 8, 128, fp8, 60, 10, seed=3)
    s.add([60, 1, 127, 300, 64])
    change = torch.ones(5, dtype=torch.int32, device="cuda")
    rows = torch.zeros((5, 48 * 128), dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.unflatten(1, (-1, 128)) for x in rows.split([32 * 128, 8 * 128, 8 * 128], dim=1))
    cu, slots = torch.empty(6, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    desc = api.make_desc(s.seq, s.table, 1, 32, 1, 60)
    ws = torch.empty(api.dsa_gqa_decode_workspace_bytes(desc, 8, 128), dtype=torch.uint8, device="cuda")
    qc, out = torch.empty((5, 32, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((5, 32, 128), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.dsa_pages_update(change, s.seq, s.table, s.free, s.count, cu, slots)
        qc.copy_(q)
        if fp8:
            api.dsa_kv_write_fp8(k, v, slots, s.caches[0], s.scales[0], s.caches[1], s.scales[1])
            api.dsa_gqa_decode_fp8kv(desc, qc, s.caches[0], s.scales[0], s.caches[1], s.scales[1], out, ws, 128 ** -0.5)
        else:
            api.dsa_kv_write(k, v, slots, *s.caches)
            api.dsa_gqa_decode(desc, qc, *s.caches, out, ws, 128 ** -0.5)
    for step in range(6):
        rows.copy_(torch.randn(rows.shape, generator=s.g, device="cuda"))
        for r in range(5):
            s.k[r], s.v[r] = torch.cat([s.k[r], k[r:r + 1]]), torch.cat([s.v[r], v[r:r + 1]])
        graph.replay()
        _near(out, s.prompt(torch.arange(6, dtype=torch.int32, device="cuda"), q, 1), fp8)
    assert s.seq.tolist() == [66, 7, 133, 306, 70] and api.dsa_get_device_error() == 0
