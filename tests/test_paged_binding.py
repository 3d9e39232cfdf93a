"""The Python binding of the paged calls without a device: what a call says of
its caches is its own, whatever other host threads do with the same plan."""
import threading

import torch


class FakeLibrary:
    """Takes a call's arguments once both threads have prepared theirs."""

    def __init__(self, threads):
        self.gate = threading.Barrier(threads)
        self.seen = {}

    def markov_paged_plan_create(self, desc, out):
        return 0

    def markov_paged_plan_destroy(self, plan):
        pass

    def _take(self, k_view, v_view):
        self.gate.wait(10)
        self.seen[threading.current_thread().name] = (k_view._obj.data, v_view._obj.data, k_view._obj.num_pages)
        self.gate.wait(10)
        return 0

    def markov_paged_write(self, plan, k, k0, k1, v, v0, v1, k_view, v_view, *rest):
        return self._take(k_view, v_view)

    def markov_paged_attention(self, plan, q, q0, q1, k_view, v_view, *rest):
        return self._take(k_view, v_view)


def test_two_threads_on_one_plan_describe_their_own_caches(monkeypatch):
    """One thread per layer, say: a layer's keys must not go to another's cache."""
    from draft_token_markov_gb300 import api
    fake = FakeLibrary(2)
    monkeypatch.setattr(api, "lib", lambda: fake)
    monkeypatch.setattr(api, "_dev", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(api, "_flat", lambda t, dtype, n, name: t.data_ptr())
    monkeypatch.setattr(api, "_stream", lambda stream: None)
    plan = api.PagedPlan(2, 2, 64, 16, device=0)
    caches = {f"layer{i}": [torch.zeros((3 + i, 16, 2, 64), dtype=torch.bfloat16) for _ in range(2)] for i in range(2)}
    new = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int64)

    def write(kc, vc):
        api.markov_paged_write(plan, new, new, kc, vc, ints)

    def attend(kc, vc):
        api.markov_paged_attention(plan, new, kc, vc, ints.view(1, 2).int(), ints[:1], ints, ints[:1], out=new.clone())

    for calls in ((write, write), (write, attend)):
        fake.seen.clear()
        threads = [threading.Thread(target=call, args=caches[name], name=name) for call, name in zip(calls, caches)]
        for t in threads:
            t.start()
        for t in threads:
            t.join(20)
        for name, (kc, vc) in caches.items():
            assert fake.seen[name] == (kc.data_ptr(), vc.data_ptr(), kc.shape[0]), name
    plan.close()
