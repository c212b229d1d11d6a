"""Host threads that decode with weights of different widths at once: each
call's launch takes its own amount of shared memory, whatever the others do."""
import threading

import pytest
import torch

from mqtest import ensure_built
from nvfp4_quantized_prefill_b200 import binding as mq
from nvfp4_quantized_prefill_b200 import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("M", [1, 2])
def test_host_threads_decode_weights_of_different_widths(M):
    N, cases = 256, []
    for i, K in enumerate((1024, 14336 // M, 2048, 8192 // M)):
        w = workloads.weight(N, K, 0.02, 31, i)
        x = workloads.activation("outlier", M, K, 31, 10 + i)
        W, xd = mq.Weight(w.cuda()), x.cuda()
        nb = mq.mq_workspace_bytes(M, K)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        alone, y = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mq.mq_decode_linear_nvfp4(W.handle, xd, M, alone, ws, nb)
        cases.append((W, xd, alone, y, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    decode, codes, go = mq.lib().mq_decode_linear_nvfp4, {}, threading.Barrier(len(cases))

    def work(i, W, x, y, ws, s):
        go.wait(30)
        codes[i] = {decode(W.handle, x.data_ptr(), M, y.data_ptr(), ws.data_ptr(), ws.numel(), s.cuda_stream)
                    for _ in range(6000)}
    threads = [threading.Thread(target=work, args=(i, c[0], c[1], c[3], c[4], c[5])) for i, c in enumerate(cases)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == {i: {0} for i in range(len(cases))}, {i: [mq.STATUS[c] for c in v] for i, v in codes.items()}
    for W, _, alone, y, _, _ in cases:
        assert torch.equal(y, alone)
        W.free()
    assert mq.mq_check() == 0
