"""What the kernels promise of their reads and no run shows, looked up in their
sources."""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "draft_token_markov_gb300", "csrc")


def _body(name, begin, end):
    """A source's text between the first occurrences of two lines' beginnings."""
    text = open(os.path.join(CSRC, name)).read()
    at = text.index(begin)
    return text[at:text.index(end, at)]


def test_logits_of_a_row_that_is_left_out_are_not_read():
    """A read of memory that need not be there: the kernel leaves before any of its
    loads of logits."""
    body = _body("logprobs.cu", "uint4 x[kTurn], y[kTurn];", " the stream\n")
    leave = body.index("if (token64 < 0 || token64 >= a.vocab) return;")
    assert leave < body.index("load(x, 0)") and "load" not in body[:leave].replace("before the first load", "")


def test_scales_of_a_tile_are_written_by_the_warp_whose_barrier_its_scores_wait_for():
    """The softmax reads a tile's scales, of keys and of values, once its scores are done;
    those wait for the keys' barrier alone, so the warp that arrives there after its
    stores has to have made them all."""
    body = _body("paged_e4m3_attention.cu", "key / value loads", "MMA issue")
    guard = body.index("if (!values && ")
    at, arrive = body.index("= scales + "), body.index("mbar_expect_tx(full")
    assert guard < at < body.index("__syncwarp();", at) < arrive and body.count("= scales + ") == 1
    text = open(os.path.join(CSRC, "paged_e4m3_attention.cu")).read()
    assert text.count("= scales + ") == 2                # the other is the softmax's


def test_a_rotary_plans_frequencies_have_arrived_when_it_is_there():
    """A copy from pageable memory may return before it is done, and a call's stream need
    not wait for the default one."""
    body = _body("rotary.cu", "markov_status markov_rotary_plan_create", "markov_status markov_rotary(")
    assert body.index("cudaMemcpy(p->turns") < body.index("cudaStreamSynchronize(nullptr)") < body.index("*out = p;")


def test_a_blocks_old_scale_is_read_before_a_thread_writes_the_new_one():
    """By a thread block behind its barrier, by a warp behind its own."""
    body = _body("paged_e4m3.cu", "__device__ __forceinline__ void store_run(", "if (tid == 0) *scale = s;")
    read = body.index("old = __ldcg(scale)")
    both = body[body.index("if (TEAM > 32) {", read):body.index("float s = scale_of(", read)]
    block, warp = both.split("} else {")
    assert "__syncthreads();" in block and "__syncwarp();" in warp
