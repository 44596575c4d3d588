"""Threads that call every operator at once, each on a stream of its own: the
bits of the same calls alone.  Their backwards share the library's stream."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def bf16(*shape, sigma=1.0):
    return (torch.randn(*shape, device="cuda") * sigma).to(torch.bfloat16)


class Job:
    def __init__(self, seed, M, K, N, r):
        import bit_nf4_quantized_pack_b200 as q
        torch.manual_seed(seed)
        self.q, self.st = q, q.new_status()
        self.w = [q.quantize(bf16(K, N, sigma=0.02)) for _ in range(2)]
        self.A, self.B = [bf16(K, r, sigma=0.02) for _ in range(2)], [bf16(r, N, sigma=0.02) for _ in range(2)]
        self.X, self.dH, self.y = bf16(M, K), bf16(M, N), torch.randint(N, (M,), device="cuda")
        self.want = [t.clone() for t in self.run()]
        torch.cuda.synchronize()

    def run(self):
        q, X, st = self.q, self.X, self.st
        args = (self.w[0], self.w[1], self.A[0], self.B[0], self.A[1], self.B[1], 2.0)
        H, saved = q.gated_forward(X, *args, save="int8", status=st)
        x8 = q.act8_quantize(X, status=st)
        grads = q.gated_backward(self.dH, x8, saved, *args, status=st)
        layer = q.linear_backward(self.dH, x8, saved.Zg, self.w[0], self.A[0], self.B[0], 2.0,
                                  grad_dtype=torch.bfloat16, status=st)
        loss, lse = q.head_loss_forward(X, self.w[1], self.y, status=st)
        return [H, *grads, *layer, loss, lse, q.head_loss_backward(loss, X, lse, self.w[1], self.y, status=st)]


def test_threads_on_their_own_streams():
    jobs = [Job(i, *s) for i, s in enumerate(((1, 4096, 2752, 16), (40, 256, 320, 5), (300, 1088, 4096, 12),
                                              (1030, 1088, 11008, 16), (1500, 4096, 2752, 64)))]
    wrong = []

    def work(i, job):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(12):
                    out = job.run()
                    stream.synchronize()
                    wrong.extend((i, k) for k, (a, b) in enumerate(zip(out, job.want)) if not torch.equal(a, b))
                if job.q.status_sync(job.st) != (0, 0):
                    wrong.append((i, "status"))
        except Exception as e:                 # noqa: BLE001  (reported below)
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=a) for a in enumerate(jobs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:10]
