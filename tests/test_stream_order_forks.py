"""The forks' second kernel starts beside the first and does not wait for it before it reads. What kernels before both wrote is
visible to it only through the word that the first one stores behind its own wait: a property of the sources, as the plain
loads behind a wait are."""
from test_stream_order import code, kernels


def body(file, name):
    return next(b for n, _, b in kernels(code(file)) if n == name)


def test_nothing_is_read_before_a_wait_or_the_word():
    text = body("paged_decode.cuh", "decode_kernel")
    head = text[:text.index("entry_of(")]
    assert "see_inputs(p);\n  else\n    pdl_wait();" in head, "every variant waits, or acquires the word, before it reads the batch"
    assert "p." not in head[:head.index("see_inputs")].replace("p.Hkv", "").replace("p.G", "")


def test_the_word_is_stored_behind_the_wait_and_before_the_second_kernel_may_start():
    text = body("paged_tile.cuh", "paged_attn_kernel")
    assert text.index("pdl_wait();") < text.index("hand_inputs_on(p)") < text.index("pdl_trigger();")


def test_the_word_is_taken_back_on_every_path():
    text = body("paged_decode.cuh", "decode_kernel")
    done = text[text.index("auto prefix_done"):]
    assert done.index("pdl_wait();") < done.index("take_word_back(p)")
    after = done[done.index("};"):]
    assert after.count("prefix_done();") == 2 and "pdl_wait" not in after


def test_store_and_load_are_a_release_and_an_acquire():
    text = code("paged.cuh")
    assert "st.release.gpu" in text[text.index("hand_inputs_on"):text.index("see_inputs")]
    seen = text[text.index("void see_inputs"):text.index("take_word_back")]
    assert "ld.acquire.gpu" in seen and "pdl_wait()" in seen and "fence.proxy.async" in seen
