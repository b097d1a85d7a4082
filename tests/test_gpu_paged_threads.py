"""One cache, two host threads, one stream: the two launches of a decode call stay together."""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_decode_attention_oasis_gb300 import build

    build.build()


def test_two_threads_decode_on_one_stream():
    """Equal ranges: pieces of pairs that cross thread blocks wait in the stream's scratch for the second
    launch.  The threads' contexts differ, so their pieces lie in different places."""
    from paged_helpers import bf16, cache_of, ints, random_pages, shuffled_table

    rng = np.random.default_rng(0)
    held, nb_max, hkv, hq, calls = [3000, 900, 40], 4000, 2, 8, 1500
    n_pages = sum(-(-n // 16) for n in held)
    kv, scale = random_pages(rng, n_pages, hkv)
    c = cache_of(kv, scale, shuffled_table(rng, held, nb_max, n_pages), hq)
    work = [(bf16(rng, (3, hq, 128))[0], ints(ctx)) for ctx in (held, [17, 900, 33])]
    want = [c.decode(q, ctx).clone() for q, ctx in work]
    torch.cuda.synchronize()
    outs, failed, start = [[], []], [], threading.Barrier(2)

    def loop(i):
        try:
            q, ctx = work[i]
            start.wait()
            for _ in range(calls):
                outs[i].append(c.decode(q, ctx))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        wrong = (torch.stack(outs[i]) != want[i]).flatten(1).any(1).sum()
        assert int(wrong) == 0, f"thread {i}: {int(wrong)} of {calls} outputs differ"
