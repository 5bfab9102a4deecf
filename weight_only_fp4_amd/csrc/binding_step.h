// The calls around a decode step's layers; part of binding.cpp, whose helpers
// they use.

// A workspace: `o`, or `need` new bytes, the first `zeros` of them cleared.
at::Tensor workspace_of(PyObject* o, int64_t need, int64_t zeros, c10::Device dev) {
    if (o != Py_None) {
        const at::Tensor& t = tensor(o, "workspace_buf");
        TORCH_CHECK_VALUE(t.device() == dev && t.is_contiguous(), "workspace_buf must be a contiguous tensor on ", dev);
        return t;
    }
    if (need < 0) check(NVFP4_ERR_INVALID_ARG);
    at::Tensor ws = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(dev));
    if (zeros > 0 && need > 0) ws.narrow(0, 0, zeros).zero_();
    return ws;
}

const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
int32_t* ints_out(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// `n` values of `base` from place `from` on, which it moves past them and the
// rest of 16 bytes: a small call's outputs are one allocation (six cost 4 us).
at::Tensor part_of(const at::Tensor& base, int64_t& from, int64_t n) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), base.dtype());
    c10::TensorImpl* impl = t.unsafeGetTensorImpl();
    impl->set_storage_offset(from);
    impl->set_sizes_contiguous({n});
    from += (n + 3) / 4 * 4;
    return t;
}

// kv_plan(cached, new, page_table, free_pages, head, page_size, tokens, out)
// -> (slots, positions, requests, lengths, offsets, head)
PyObject* kv_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& cached = tensor(a[0], "cached");
    TORCH_CHECK_VALUE(cached.scalar_type() == at::kInt && cached.dim() == 1 && cached.is_cuda(),
                      "cached must be a 1-d int32 tensor on the GPU");
    unit_stride(cached, "cached");
    const c10::Device dev = cached.device();
    c10::DeviceGuard guard(dev);
    const int64_t B = cached.size(0);
    const at::Tensor& fresh_tokens = same(a[1], "new", at::kInt, {B}, dev);
    const at::Tensor& table = tensor(a[2], "page_table");
    TORCH_CHECK_VALUE(table.dim() == 2 && table.size(0) == B, "page_table must be an int32 tensor [", B, ", max_pages]");
    same(a[2], "page_table", at::kInt, table.sizes(), dev);
    own_rows(table, "page_table");
    const at::Tensor& list = tensor(a[3], "free_pages");
    TORCH_CHECK_VALUE(list.dim() == 1, "free_pages must be a 1-d int32 tensor");
    same(a[3], "free_pages", at::kInt, list.sizes(), dev);
    const at::Tensor& head = same(a[4], "free_head", at::kInt, {1}, dev);
    const int64_t page = whole(a[5]), T = whole(a[6]);
    TORCH_CHECK_VALUE(T >= 0, "tokens must not be negative, got ", T);
    PyObject* given[6] = {Py_None, Py_None, Py_None, Py_None, Py_None, Py_None};
    if (a[7] != Py_None) {
        TORCH_CHECK_VALUE(PyTuple_Check(a[7]) && PyTuple_GET_SIZE(a[7]) == 6,
                          "out must be a plan, or six tensors (slots, positions, requests, lengths, offsets, head)");
        for (int i = 0; i < 6; ++i) given[i] = PyTuple_GET_ITEM(a[7], i);
    }
    const char* names[6] = {"slots", "positions", "requests", "lengths", "offsets", "head"};
    const int64_t sizes[6] = {T, T, T, B, B + 1, 1};
    const int64_t need = nvfp4_kv_plan_workspace_bytes(B, T);
    if (need < 0) check(NVFP4_ERR_INVALID_ARG);
    at::Tensor out[6], ws;
    if (a[7] == Py_None) {
        int64_t total = need / 4, from = 0;
        for (int64_t n : sizes) total += (n + 3) / 4 * 4;
        const at::Tensor all = fresh({total}, at::kInt, dev);
        for (int i = 0; i < 6; ++i) out[i] = part_of(all, from, sizes[i]);
        ws = part_of(all, from, need / 4);
    } else {
        for (int i = 0; i < 6; ++i) out[i] = output(given[i], names[i], at::kInt, {sizes[i]}, dev);
        ws = workspace_of(Py_None, need, 0, dev);
    }
    check(nvfp4_kv_plan(ints(cached), ints(fresh_tokens), B, ints_out(table), leading(table), table.size(1), page, ints(list),
                        list.size(0), ints(head), T, ints_out(out[0]), ints_out(out[1]), ints_out(out[2]), ints_out(out[3]),
                        ints_out(out[4]), ints_out(out[5]), ws.data_ptr(), need, stream_of(dev)));
    PyObject* t = PyTuple_New(6);
    if (!t) throw python_error();
    for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(std::move(out[i])));
    return t;
    END_HANDLE_TH_ERRORS
}

// Strides of a stack of matrices [L, rows, columns].
void matrices(const at::Tensor& t, int64_t (&stride)[2]) {
    stride[0] = step(t, 0);
    stride[1] = step(t, 1);
}

// lora_add(y, x, a, b, adapter, scale, out, workspace) -> out
PyObject* lora_add(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const at::Tensor& x = act(a[1], "x", 2);
    const at::ScalarType type = x.scalar_type();
    const c10::Device dev = x.device();
    c10::DeviceGuard guard(dev);
    const int64_t T = x.size(0), K = x.size(1);
    const at::Tensor& y = tensor(a[0], "y");
    TORCH_CHECK_VALUE(y.dim() == 2, "y must have 2 dims, got shape ", y.sizes());
    const int64_t N = y.size(1);
    same(a[0], "y", type, {T, N}, dev);
    const at::Tensor& A = act(a[2], "a", 3);
    const int64_t L = A.size(0), R = A.size(1);
    same(a[2], "a", type, {L, R, K}, dev);
    const at::Tensor& Bm = same(a[3], "b", type, {L, N, R}, dev);
    const at::Tensor& adapter = same(a[4], "adapter", at::kInt, {T}, dev);
    const float* scale = a[5] == Py_None ? nullptr : static_cast<const float*>(same(a[5], "scale", at::kFloat, {L}, dev).data_ptr());
    at::Tensor out = output(a[6], "out", type, {T, N}, dev);
    const int64_t need = nvfp4_lora_workspace_bytes(T, K, N, R);
    at::Tensor ws = workspace_of(a[7], need, 0, dev);
    int64_t sa[2], sb[2];
    matrices(A, sa);
    matrices(Bm, sb);
    check(nvfp4_lora_add(x.data_ptr(), leading(x), A.data_ptr(), sa[0], sa[1], Bm.data_ptr(), sb[0], sb[1], ints(adapter), scale,
                         y.data_ptr(), leading(y), out.data_ptr(), leading(out), T, K, N, R, L, ws.data_ptr(),
                         (int64_t)ws.nbytes(), type == at::kHalf, stream_of(dev)));
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

const void* blob_of(PyObject* o, const char* name, int64_t bytes, c10::Device dev) {
    const at::Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kByte && t.is_contiguous() && t.device() == dev, name,
                      " must be a contiguous uint8 tensor on ", dev);
    TORCH_CHECK_VALUE(bytes < 0 || t.numel() >= bytes, name, " has ", t.numel(), " bytes, the repacked weights of this shape ", bytes);
    return t.data_ptr();
}

// moe_layer(x, topk_ids, topk_weights, w1, w2, E, I, g1, g2, divisor, activation, pre_scale1, pre_scale2, mxfp4, out, workspace)
// -> out
PyObject* moe_layer(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 16);
    const at::Tensor& x = act(a[0], "x", 2);
    const at::ScalarType type = x.scalar_type();
    const c10::Device dev = x.device();
    c10::DeviceGuard guard(dev);
    const int64_t T = x.size(0), H = x.size(1);
    const at::Tensor& ids = tensor(a[1], "topk_ids");
    TORCH_CHECK_VALUE(ids.dim() == 2 && ids.size(0) == T && ids.is_contiguous(), "topk_ids must be a contiguous int32 tensor [", T,
                      ", k]");
    const int64_t k = ids.size(1);
    same(a[1], "topk_ids", at::kInt, {T, k}, dev);
    const at::Tensor& weights = same(a[2], "topk_weights", at::kFloat, {T, k}, dev);
    TORCH_CHECK_VALUE(weights.is_contiguous(), "topk_weights must be contiguous");
    const int64_t E = whole(a[5]), I = whole(a[6]), activation = whole(a[10]);
    const bool mx = truth(a[13]);
    const int64_t need = nvfp4_moe_layer_workspace_bytes(T, k, E, H, I);
    if (need < 0) check(NVFP4_ERR_INVALID_ARG);
    const bool gated = activation == NVFP4_MOE_SILU_GLU;
    const void* w1 = blob_of(a[3], "w1", gated ? nvfp4_repack_gated_bytes(E, I, H) : nvfp4_repack_bytes(E, I, H), dev);
    const void* w2 = blob_of(a[4], "w2", nvfp4_repack_bytes(E, H, I), dev);
    auto per_expert = [&](PyObject* o, const char* name) {
        return o == Py_None ? nullptr : static_cast<const float*>(same(o, name, at::kFloat, {E}, dev).data_ptr());
    };
    auto per_column = [&](PyObject* o, const char* name, int64_t columns) {
        return o == Py_None ? nullptr : same(o, name, type, {columns}, dev).data_ptr();
    };
    const float *g1 = per_expert(a[7], "g1"), *g2 = per_expert(a[8], "g2");
    const void *p1 = per_column(a[11], "pre_scale1", H), *p2 = per_column(a[12], "pre_scale2", I);
    at::Tensor out = output(a[14], "out", type, {T, H}, dev);
    at::Tensor ws = workspace_of(a[15], need, NVFP4_MOE_LAYER_COUNTER_BYTES, dev);
    check(nvfp4_moe_layer(x.data_ptr(), leading(x), ints(ids), static_cast<const float*>(weights.data_ptr()), T, k, p1, w1, g1,
                          p2, w2, g2, truth(a[9]), (int)activation, out.data_ptr(), leading(out), E, H, I, ws.data_ptr(),
                          (int64_t)ws.nbytes(), type == at::kHalf, mx, stream_of(dev)));
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// sample(logits, u, temperature, top_k, top_p, min_p, return_logprobs, out, workspace) -> tokens or (tokens, logprobs)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 9);
    const at::Tensor& l = tensor(a[0], "logits");
    TORCH_CHECK_VALUE(l.is_cuda() && l.dim() == 2 && (is_act(l.scalar_type()) || l.scalar_type() == at::kFloat),
                      "logits must be a bf16, fp16 or fp32 tensor [rows, vocabulary] on the GPU");
    unit_stride(l, "logits");
    const c10::Device dev = l.device();
    c10::DeviceGuard guard(dev);
    const int64_t B = l.size(0), V = l.size(1);
    auto row = [&](PyObject* o, const char* name) {
        return o == Py_None ? nullptr : static_cast<const float*>(same(o, name, at::kFloat, {B}, dev).data_ptr());
    };
    const at::Tensor& u = same(a[1], "u", at::kFloat, {B}, dev);
    const float *t = row(a[2], "temperature"), *p = row(a[4], "top_p"), *mp = row(a[5], "min_p");
    const int32_t* k = a[3] == Py_None ? nullptr : ints(same(a[3], "top_k", at::kInt, {B}, dev));
    const bool want = truth(a[6]);
    at::Tensor tokens = output(a[7], "out", at::kInt, {B}, dev), logprobs;
    if (want) logprobs = fresh({B}, at::kFloat, dev);
    at::Tensor ws = workspace_of(a[8], nvfp4_sample_workspace_bytes(B, V), 0, dev);
    const int type = l.scalar_type() == at::kFloat ? NVFP4_LOGITS_F32 : l.scalar_type() == at::kHalf ? NVFP4_LOGITS_F16 : NVFP4_LOGITS_BF16;
    check(nvfp4_sample(l.data_ptr(), leading(l), type, B, V, static_cast<const float*>(u.data_ptr()), t, k, p, mp,
                       ints_out(tokens), want ? static_cast<float*>(logprobs.data_ptr()) : nullptr, ws.data_ptr(),
                       (int64_t)ws.nbytes(), stream_of(dev)));
    PyObject* o = THPVariable_Wrap(std::move(tokens));
    return want ? pack({o, THPVariable_Wrap(std::move(logprobs))}) : o;
    END_HANDLE_TH_ERRORS
}
